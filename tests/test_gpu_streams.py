"""Workspaces that a call makes for itself: cleared, and given back, in the order of the stream that the call runs on."""
import pytest
import torch

from speculative_decoding_eagle_gb300 import binding as E
from speculative_decoding_eagle_gb300 import step as S
from speculative_decoding_eagle_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture
def made(monkeypatch):
    """The streams that workspaces were made on."""
    seen, make = [], E.new_workspace

    def new_workspace(*args, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return make(*args, **kw)
    monkeypatch.setattr(E, "new_workspace", new_workspace)
    return seen


def test_a_step_on_a_side_stream_clears_its_attention_workspace_there(made):
    wl = W.WORKLOADS["tiny"]
    st = S.VerifyStep(wl)
    inp = S.to_device(wl, S.host_inputs(wl, st.C))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    made.clear()
    st.run(inp, stream=side)
    assert made == [side.cuda_stream]
    st.run(inp, stream=side)  # the same shape: nothing new
    torch.cuda.synchronize()
    assert made == [side.cuda_stream] and int(st.dev_status.item()) == 0


def test_a_sampled_tree_without_a_workspace_makes_one_on_its_stream(made):
    B, V, widths = 2, 1000, (3, 2)
    parent, _ = W.static_shape(widths)
    N = parent.size
    gen = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(B * N, V, generator=gen, device="cuda")
    u = torch.rand(B, N, generator=gen, device="cuda")
    rmap = torch.arange(B * N, dtype=torch.int32, device="cuda").view(B, N)
    side = torch.cuda.Stream()
    trees = [E.TreeBuffers.allocate_flat(B, N) for _ in range(2)]
    side.wait_stream(torch.cuda.current_stream())
    for tree, stream in zip(trees, (side, None)):
        made.clear()
        E.et_static_tree_sampled(B, V, 1.0, torch.from_numpy(parent).cuda(), logits, rmap, u, tree, stream=stream)
        assert made == [(stream or torch.cuda.current_stream()).cuda_stream]
    torch.cuda.synchronize()
    assert torch.equal(trees[0].flat_tok, trees[1].flat_tok)
