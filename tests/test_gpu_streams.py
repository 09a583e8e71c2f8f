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
