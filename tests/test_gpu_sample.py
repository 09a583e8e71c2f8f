"""Sampling from truncated logits on the GPU, against the definition in 64 bits: tokens and kept sets have to be equal (the
inputs keep borders apart where a test does not put them there on purpose), log-probabilities to 4e-7 (1 + |x|): the
result is rounded once to fp32 (2^-24) from 64-bit values of weights that are good to 2^-40."""
import numpy as np
import pytest
import torch

from speculative_decoding_eagle_gb300 import binding as E

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_eagle_gb300 import build_lib
    build_lib.build()
    E.load()


def reference(z, T, k, p, m, u):
    """One row: token, log-probability, kept mask.  z fp32 numpy, settings as the fp32 / int values that the call reads."""
    z = z.astype(np.float64)
    z = np.where(np.isnan(z), -np.inf, np.where(z == np.inf, np.finfo(np.float32).max, z))
    V = len(z)
    keep = np.zeros(V, bool)
    if z.max() == -np.inf:
        return -1, -np.inf, keep
    ids = np.lexsort((np.arange(V), -z))
    ids = ids[z[ids] > -np.inf]
    if not T > 0:
        keep[ids[0]] = True
        return int(ids[0]), 0.0, keep
    if k > 0:
        ids = ids[:k]
    depth = (z[ids] - z.max()) / np.float64(T)
    w = np.exp(depth)
    if p < 1:
        before = np.cumsum(w) - w
        n = int(np.sum(before < np.float64(p) * w.sum()))
        ids, w, depth = ids[:max(n, 1)], w[:max(n, 1)], depth[:max(n, 1)]
    if m > 0:
        ok = depth >= np.log(np.float64(m))
        ok[0] = True
        ids, w = ids[ok], w[ok]
    keep[ids] = True
    order = np.argsort(ids)
    run = np.cumsum(w[order])
    u = min(max(float(u), 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    at = min(int(np.sum(run <= u * run[-1])), len(run) - 1)
    t = int(ids[order][at])
    return t, float(np.log(w[order][at] / run[-1])), keep


def call(z, T=None, k=None, p=None, m=None, u=None, want_status=0, truncated=True, stream=None):
    B, V = z.shape
    dev = lambda x, t: None if x is None else torch.as_tensor(np.asarray(x, t)).cuda()  # noqa: E731
    zt = z if isinstance(z, torch.Tensor) else torch.from_numpy(z).cuda()
    tok = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((B,), 7.0, device="cuda")
    tr = torch.full((B, V), 7.0, device="cuda") if truncated else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.et_sample(zt, dev(u, np.float32), tok, temperature=dev(T, np.float32), top_k=dev(k, np.int32),
                top_p=dev(p, np.float32), min_p=dev(m, np.float32), logprob=lp, truncated=tr, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    assert int(st.item()) == want_status
    return tok.cpu().numpy(), lp.cpu().numpy(), None if tr is None else tr.cpu().numpy()


def check(z, T=None, k=None, p=None, m=None, u=None, **kw):
    B = z.shape[0]
    tok, lp, tr = call(z, T, k, p, m, u, **kw)
    f = lambda x, d: np.full(B, d, np.float32) if x is None else np.asarray(x, np.float32)  # noqa: E731
    T, p, m, u = f(T, 1), f(p, 1), f(m, 0), f(u, 0)
    k = np.zeros(B, int) if k is None else np.asarray(k)
    for b in range(B):
        t, l, keep = reference(z[b], T[b], k[b], p[b], m[b], u[b])
        assert tok[b] == t, (b, tok[b], t, T[b], k[b], p[b], m[b], u[b])
        assert lp[b] == l or abs(lp[b] - l) <= 4e-7 * (1 + abs(l)), (b, lp[b], l)
        if tr is not None:
            want = np.where(keep, z[b], -np.inf)
            want = np.where(want == np.inf, np.finfo(np.float32).max, want)
            np.testing.assert_array_equal(tr[b], want)


def rows(B, V, seed, kind="zipf"):
    rng = np.random.default_rng(seed)
    if kind == "zipf":
        rank = np.argsort(rng.random((B, V)), 1)
        return (-1.2 * np.log(rank + 1.0) + rng.standard_normal((B, V))).astype(np.float32), rng
    if kind == "flat":
        return (0.3 * rng.standard_normal((B, V))).astype(np.float32), rng
    if kind == "bf16":  # rounded logits: many ties
        x = torch.from_numpy((2 * rng.standard_normal((B, V))).astype(np.float32)).to(torch.bfloat16).float().numpy()
        return x, rng
    if kind == "masked":  # the type's lowest value and -inf in masked places
        x = (3 * rng.standard_normal((B, V))).astype(np.float32)
        x[rng.random((B, V)) < 0.5] = -np.inf
        x[rng.random((B, V)) < 0.3] = np.finfo(np.float32).min
        x[:, 0] = 1.0
        return x, rng
    return np.full((B, V), 0.25, np.float32), rng  # "equal"


@pytest.mark.parametrize("kind", ["zipf", "flat", "bf16", "masked", "equal"])
@pytest.mark.parametrize("V", [1, 2, 31, 100, 1000, 4097, 32000, 70001])
def test_settings_of_every_row(V, kind):
    B = 24
    z, rng = rows(B, V, V, kind)
    T = rng.choice([0.0, -1.0, 0.3, 0.8, 1.0, 1.7], B)
    k = rng.choice([0, -3, 1, 2, 20, 50, 1000, 5000, V, V + 5], B)
    p = rng.choice([1.0, 1.5, 0.0, 0.1, 0.5, 0.9, 0.99], B)
    m = rng.choice([0.0, -1.0, 0.01, 0.2, 1.0, 2.0], B)
    check(z, T, k, p, m, rng.random(B, np.float32))


@pytest.mark.parametrize("V", [1000, 32000, 262144])
@pytest.mark.parametrize("B", [1, 3, 40, 200])
def test_one_setting_at_a_time(B, V):
    if B * V > 10_000_000:
        pytest.skip("the reference sorts row by row")
    z, rng = rows(B, V, B + V)
    u = rng.random(B, np.float32)
    check(z, u=u)
    check(z, T=np.full(B, 0.7), u=u)
    check(z, k=np.full(B, 40), u=u)
    check(z, k=np.full(B, 3000), u=u)
    check(z, p=np.full(B, 0.95), u=u)
    check(z, m=np.full(B, 0.05), u=u)


def test_uniforms_at_the_borders():
    # four equal weights: the borders are the quarters themselves, and a border belongs to the next token
    z = np.full((9, 4), -2.0, np.float32)
    u = np.array([0, 0.25, np.nextafter(np.float32(0.25), 0), 0.5, 0.75, np.nextafter(np.float32(1), 0), 1.0, -0.5, np.nan], np.float32)
    tok, _, _ = call(z, u=u)
    assert tok.tolist() == [0, 1, 0, 2, 3, 3, 3, 0, 0]


def test_ties_go_to_the_lowest_ids():
    z = np.zeros((1, 5000), np.float32)
    z[0, 17] = 1.0
    _, _, tr = call(z, k=[5], u=[0.5])
    assert np.flatnonzero(tr[0] > -np.inf).tolist() == [0, 1, 2, 3, 17]
    # top-p among ties: 0.4 of 5000 equal weights are the first 2000 ids; the kept share reaches it with the last of them
    z[:] = 3.0
    _, _, tr = call(z, p=[np.float32(0.4)], u=[0.5])
    n = int(np.sum(np.arange(5000) < np.float64(np.float32(0.4)) * 5000))
    assert np.flatnonzero(tr[0] > -np.inf).tolist() == list(range(n))


def test_draws_agree_with_64_bits_over_many_rows():
    """No truncation: every id is a border.  With fp32 sums some of these 4000 draws would differ."""
    z, rng = rows(500, 32000, 5, "flat")
    zt = torch.from_numpy(z).cuda()
    w = torch.exp((zt - zt.amax(1, keepdim=True)).double())
    run = torch.cumsum(w, 1)
    for s in range(8):
        u = rng.random(500, np.float32)
        tok, _, _ = call(zt, u=u, truncated=False)
        want = (run <= torch.from_numpy(u).cuda().double()[:, None] * run[:, -1:]).sum(1).cpu().numpy()
        np.testing.assert_array_equal(tok, want)


def test_nonfinite_rows():
    z, rng = rows(5, 1000, 9)
    z[0, 3] = np.nan
    z[1, 7] = np.inf
    z[2, :] = -np.inf
    z[3, :] = np.nan
    z[4, 5] = np.inf
    z[4, 900] = np.inf
    for T in (0.0, 1.0):
        check(z, T=np.full(5, T), k=[0, 0, 3, 0, 2], u=rng.random(5, np.float32), want_status=E.ET_DEV_NONFINITE)


def test_strided_rows_and_a_side_stream():
    z, rng = rows(6, 999, 11)
    big = torch.zeros(6, 1500, device="cuda")
    big[:, 3:1002] = torch.from_numpy(z).cuda()  # neither stride nor offset a multiple of 16 bytes
    u = rng.random(6, np.float32)
    want = call(torch.from_numpy(z).cuda(), k=np.full(6, 30), p=np.full(6, 0.8), u=u)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(big[:, 3:1002], k=np.full(6, 30), p=np.full(6, 0.8), u=u, stream=s)
    for a, b in zip(want, got):
        np.testing.assert_array_equal(a, b)


def test_captured_and_replayed_on_new_inputs():
    z, rng = rows(4, 32000, 13)
    zt, u = torch.from_numpy(z).cuda(), torch.rand(4, device="cuda")
    k, p = torch.full((4,), 60, dtype=torch.int32, device="cuda"), torch.full((4,), 0.9, device="cuda")
    tok, lp = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    E.et_sample(zt, u, tok, top_k=k, top_p=p, logprob=lp)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        E.et_sample(zt, u, tok, top_k=k, top_p=p, logprob=lp)
    for s in range(3):
        z, rng = rows(4, 32000, 20 + s)
        zt.copy_(torch.from_numpy(z))
        u.copy_(torch.from_numpy(rng.random(4, np.float32)))
        k.fill_(10 + 100 * s)
        g.replay()
        torch.cuda.synchronize()
        for b in range(4):
            t, l, _ = reference(z[b], 1.0, 10 + 100 * s, np.float32(0.9), 0.0, u[b].item())
            assert tok[b].item() == t and abs(lp[b].item() - l) <= 4e-7 * (1 + abs(l))


def test_acceptance_under_truncated_logits():
    """What the walk draws from the truncated rows lies in the kept sets, and greedily it is what the sampler draws."""
    B, V, n = 3, 1000, 8
    z, rng = rows(B * (n + 1), V, 31)
    N = n + 1
    zt = torch.from_numpy(z).cuda()
    tr = torch.empty_like(zt)
    tok = torch.zeros(B * N, dtype=torch.int32, device="cuda")
    u = torch.from_numpy(rng.random(B * N, np.float32)).cuda()
    T = 0.8
    E.et_sample(zt, u, tok, temperature=torch.full((B * N,), T, device="cuda"),
                top_p=torch.full((B * N,), 0.7, device="cuda"), truncated=tr)
    cfg = E.TreeCfg(B=B, V=V, depth=2, topk=4, m=4, n=n, temperature=T)
    tree = E.TreeBuffers.allocate(cfg)
    tree.flat_parent.copy_(torch.tensor([[-1, 0, 0, 0, 0, 1, 1, 2, 2]] * B, dtype=torch.int32))
    tree.flat_depth.copy_(torch.tensor([[0, 1, 1, 1, 1, 2, 2, 2, 2]] * B, dtype=torch.int32))
    tree.flat_tok.copy_(torch.argsort(-zt.view(B, N, V)[:, 0], dim=1)[:, :N].to(torch.int32))
    acc, path = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, 3, dtype=torch.int32, device="cuda")
    out = torch.zeros(B, 3, dtype=torch.int32, device="cuda")
    ws = E.new_workspace(E.et_tree_workspace_size(cfg))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.et_verify_accept(cfg, E.ET_ACCEPT_STOCH_POINT, tree, tr, acc, path, out, ws,
                       uniforms=torch.from_numpy(rng.random((B, N), np.float32)).cuda(), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    kept = (tr > float("-inf")).view(B, N, V)
    for b in range(B):
        row = 0
        for i in range(int(acc[b]) + 1):
            assert bool(kept[b, row, int(out[b, i])])
            if i < int(acc[b]):
                row = int(path[b, i + 1])
