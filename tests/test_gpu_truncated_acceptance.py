"""The acceptance walk on truncated logits: greedy rows give the sampler's tokens, and over many draws the first token has the
distribution of the truncated softmax."""
import numpy as np
import pytest
import torch

from speculative_decoding_eagle_gb300 import binding as E

pytestmark = pytest.mark.gpu
PARENT = [-1, 0, 0, 0, 0, 1, 1, 2, 2]
DEPTH = [0, 1, 1, 1, 1, 2, 2, 2, 2]
N = len(PARENT)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_eagle_gb300 import build_lib
    build_lib.build()
    E.load()


def make_tree(B, V, T, tokens):
    cfg = E.TreeCfg(B=B, V=V, depth=2, topk=4, m=4, n=N - 1, temperature=T)
    tree = E.TreeBuffers.allocate(cfg)
    tree.flat_parent.copy_(torch.tensor([PARENT] * B, dtype=torch.int32))
    tree.flat_depth.copy_(torch.tensor([DEPTH] * B, dtype=torch.int32))
    tree.flat_tok.copy_(tokens.to(torch.int32))
    return cfg, tree


def accept(cfg, tree, mode, target, uniforms=None):
    B = cfg.B
    acc, path = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, 3, dtype=torch.int32, device="cuda")
    out = torch.zeros(B, 3, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = E.new_workspace(E.et_tree_workspace_size(cfg))
    E.et_verify_accept(cfg, mode, tree, target, acc, path, out, ws, uniforms=uniforms, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return acc.tolist(), path.tolist(), out.tolist()


@pytest.mark.parametrize("B", [3, 12])  # every row read at once; the accepted path walked
def test_greedy_rows_give_the_samplers_tokens(B):
    V = 1000
    g = torch.Generator(device="cuda").manual_seed(41)
    z = torch.randn(B * N, V, generator=g, device="cuda")
    z[:, 17] = z[:, 900] = z.amax(1) * 1.01 + 1                       # a tie: the lower id
    z[::3, 400] = z[::3, 17] + 1
    tok = torch.full((B * N,), -7, dtype=torch.int32, device="cuda")
    tr = torch.full_like(z, 7.0)
    E.et_sample(z, torch.rand(B * N, generator=g, device="cuda"), tok, temperature=torch.zeros(B * N, device="cuda"), truncated=tr)
    assert bool(((tr > float("-inf")).sum(1) == 1).all()) and torch.equal(torch.argmax(tr, 1).int(), tok)
    assert set(tok.tolist()) == {17, 400}
    best = tok.view(B, N)
    # sequence b accepts b % 3 tokens: child 2 of the root is its token, and row 7, a child of row 2, is row 2's
    tokens = torch.arange(500, 500 + N, device="cuda").repeat(B, 1)
    b = torch.arange(B, device="cuda")
    tokens[:, 2] = torch.where(b % 3 >= 1, best[:, 0].long(), tokens[:, 2])
    tokens[:, 7] = torch.where(b % 3 == 2, best[:, 2].long(), tokens[:, 7])
    uniforms = torch.rand(B, N, generator=g, device="cuda")
    for T in (1.0, 0.3):
        cfg, tree = make_tree(B, V, T, tokens)
        for mode, u in ((E.ET_ACCEPT_GREEDY, None), (E.ET_ACCEPT_STOCH_POINT, uniforms)):
            acc, path, out = accept(cfg, tree, mode, tr, u)
            for b in range(B):
                assert acc[b] == b % 3
                rows = [0, 2, 7][:acc[b] + 1]
                assert path[b][:acc[b] + 1] == rows
                assert out[b][:acc[b] + 1] == [int(best[b, r]) for r in rows]


def test_first_tokens_have_the_truncated_distribution():
    """4096 walks over one tree.  A frequency of 4096 draws is within five standard deviations, sqrt(p (1 - p) / 4096), of its
    share (one in 10^6 falls outside) and half a draw."""
    B, V, T = 4096, 200, 0.8
    rng = np.random.default_rng(43)
    row = torch.from_numpy((2 * rng.standard_normal(V)).astype(np.float32)).cuda()
    z = row.repeat(B * N, 1)
    tr = torch.empty_like(z)
    tok = torch.zeros(B * N, dtype=torch.int32, device="cuda")
    u = lambda *s: torch.from_numpy(rng.random(s, np.float32)).cuda()  # noqa: E731
    full = lambda x: torch.full((B * N,), x, device="cuda")  # noqa: E731
    E.et_sample(z, u(B * N), tok, temperature=full(T), top_p=full(0.8), truncated=tr)
    want = torch.softmax(tr[0].double() / T, 0).cpu().numpy()
    kept = np.flatnonzero(want)
    assert 5 < len(kept) < 100
    order = torch.argsort(-row)
    # children of the root: the largest token, one in the middle of the kept set, one that is left out, the second largest
    tokens = torch.zeros(B, N, dtype=torch.int64, device="cuda")
    tokens[:, 1:5] = torch.stack([order[0], order[len(kept) // 2], order[len(kept) + 3], order[1]])
    tokens[:, 5:] = order[2:6]
    cfg, tree = make_tree(B, V, T, tokens)
    acc, _, out = accept(cfg, tree, E.ET_ACCEPT_STOCH_POINT, tr, u(B, N))
    first = np.bincount([o[0] for o in out], minlength=V) / B
    share = np.bincount(tok.cpu().numpy(), minlength=V) / (B * N)  # the sampler's own draws, nine times as many
    assert first[want == 0].sum() == 0 and share[want == 0].sum() == 0
    dev = np.sqrt(want * (1 - want))
    assert np.all(np.abs(first - want) <= 5 * dev / np.sqrt(B) + 0.5 / B)
    assert np.all(np.abs(share - want) <= 5 * dev / np.sqrt(B * N) + 0.5 / (B * N))
    assert 0 < sum(a > 0 for a in acc) < B and max(acc) == 2
