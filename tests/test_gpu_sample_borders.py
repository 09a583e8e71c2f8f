"""Sampling where more tokens than one block sorts lie in the border's step of the first histogram, thousands of distinct
logits among them: the histograms over the logits' keys find the border, in up to four rounds.  Against 64 bits, as in
test_gpu_sample; that a row takes this way is checked first, on the CPU."""
import numpy as np
import pytest
import torch

from speculative_decoding_eagle_gb300 import binding as E
from test_gpu_sample import check, reference

BINS, LIST = 512, 1024  # steps of the first histogram; tokens that one block sorts
T = 10.0                # the tokens far below the largest hold most of the mass


def dense(kind, V, seed):
    """A row with one logit of 30 that stretches the steps over tokens that lie close together."""
    rng = np.random.default_rng(seed)
    z = (0.001 * rng.standard_normal(V)).astype(np.float32)      # both signs: keys across every exponent
    if kind == "ulps":                                           # 6000 neighbouring values of one exponent
        z = (np.float32(-3.0).view(np.int32) - rng.integers(0, 6000, V).astype(np.int32)).view(np.float32)
    if kind == "ties":                                           # some 2000 values, zeros of both signs among them
        z = (np.round(rng.standard_normal(V) * 300) / np.float32(2 ** 18)).astype(np.float32)
        z[rng.random(V) < 0.01] = -0.0
    if kind == "two":                                            # many tokens above the border's step
        z[rng.random(V) < 0.4] += np.float32(2.0)
    if kind == "masked":
        z[rng.random(V) < 0.3] = -np.inf
        z[rng.random(V) < 0.1] = np.finfo(np.float32).min
    z[int(rng.integers(V))] = 30.0
    return z


def step_sizes(z, keep_before, last):
    """Tokens and distinct logits in the step that token `last` lies in, of those in keep_before."""
    f = np.float32
    top = z.max()
    width = min(f(top - z[z > -np.inf].min()), f(max(32 * T, 32)))
    with np.errstate(over="ignore"):
        step = np.minimum(BINS - 1, ((top - z) * f(f(BINS - 1) / width)).clip(0, 1e9))
    step = np.where(z > -np.inf, step, -1).astype(np.int64)
    here = keep_before & (step == step[last])
    return int(here.sum()), len(np.unique(z[here]))


def goes_through_the_keys(z, k, p):
    """Does each border that the settings ask for lie in a step of more tokens than one block sorts, and enough values?"""
    live = z > -np.inf
    order = np.lexsort((np.arange(len(z)), -z.astype(np.float64)))[:int(live.sum())]
    ok = True
    if k:
        n, values = step_sizes(z, live, order[k - 1])
        ok = ok and n > LIST and values > BINS
        order = order[:k]
        live = np.zeros(len(z), bool)
        live[order] = True
    if p < 1:
        kept = reference(z, np.float32(T), k, np.float32(p), 0.0, 0.5)[2]
        last = order[int(kept.sum()) - 1]
        n, values = step_sizes(z, live, last)
        ok = ok and n > LIST and values > BINS
    return ok


KINDS = ["normal", "ulps", "ties", "two"]
SIZES = [(1, 32000), (1, 262144), (80, 20000), (100, 50001)]  # eight blocks a row, twice; one; four
SETTINGS = [(0.55, 1.0), (0.8, 1.0), (0, 0.45), (0, 0.8), (0.9, 0.75)]  # top_k as a share of the row, top_p


def cases(kind, B, V):
    rows = min(B, 4)  # the reference sorts row by row: a batch repeats these
    z = [dense(kind, V, 1000 * V + r) for r in range(rows)]
    return [(z, int(share * V), p) for share, p in SETTINGS]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,V", SIZES)
def test_the_rows_take_this_way(B, V, kind):
    for z, k, p in cases(kind, B, V):
        assert all(goes_through_the_keys(row, k, p) for row in z)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,V", SIZES)
def test_borders_among_many_close_logits(B, V, kind):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_eagle_gb300 import build_lib
    build_lib.build()
    rng = np.random.default_rng(V)
    for z, k, p in cases(kind, B, V):
        n = len(z)
        u = rng.random(n, np.float32)
        if B == n:
            check(np.stack(z), T=np.full(n, T), k=np.full(n, k), p=np.full(n, p), u=u)
            continue
        check_repeated(z, B, k, p, u)


def check_repeated(z, B, k, p, u):
    """The rows of a batch repeat a few: these are compared with the definition, the others with them."""
    n = len(z)
    V = len(z[0])
    tile = lambda x: x.repeat((B + n - 1) // n, *([1] * (x.dim() - 1)))[:B].contiguous()  # noqa: E731
    zt, ut = tile(torch.from_numpy(np.stack(z)).cuda()), tile(torch.from_numpy(u).cuda())
    full = lambda x, t: torch.full((B,), x, dtype=t, device="cuda")  # noqa: E731
    tok, lp, tr = full(-7, torch.int32), full(7.0, torch.float32), torch.full((B, V), 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.et_sample(zt, ut, tok, temperature=full(T, torch.float32), top_k=full(k, torch.int32), top_p=full(p, torch.float32),
                logprob=lp, truncated=tr, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for r in range(n):
        t, l, keep = reference(z[r], np.float32(T), k, np.float32(p), 0.0, u[r])
        assert int(tok[r]) == t and abs(float(lp[r]) - l) <= 4e-7 * (1 + abs(l))
        np.testing.assert_array_equal(tr[r].cpu().numpy(), np.where(keep, z[r], -np.inf))
    for x in (tok, lp, tr):
        assert torch.equal(x, tile(x[:n]))


@pytest.mark.gpu
@pytest.mark.parametrize("B,V", [(1, 40000), (90, 20000)])
def test_masked_tokens_and_min_p_beside_the_borders(B, V):
    """-inf and the type's lowest value in the last step, a top_k past the tokens that are there, min_p inside the step."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rng = np.random.default_rng(7)
    rows = min(B, 3)
    z = np.stack([dense("masked", V, 50 + r) for r in range(rows)])
    inside = np.float32(np.exp(-3.00002))
    for k, p, m in ((V // 3, 1.0, 0.0), (V - 1, 0.8, 0.0), (0, 0.999, 0.0), (V // 2, 1.0, inside), (0, 0.9, inside), (V // 2, 0.9, inside)):
        zz = np.concatenate([z] * (B // rows))
        check(zz, T=np.full(len(zz), T), k=np.full(len(zz), k), p=np.full(len(zz), p), m=np.full(len(zz), m),
              u=rng.random(len(zz), np.float32))
