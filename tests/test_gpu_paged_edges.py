"""The paged cache's calls at the edges of what they accept: extreme head counts, lengths next to 2^31, values that are
not finite, handles that are copied."""
import copy
import math

import numpy as np
import pytest
import torch

import oracle as O
from speculative_decoding_eagle_gb300 import binding as E
from tests.test_gpu_paged import Pool, check_all, random_tree, run_attention

pytestmark = pytest.mark.gpu


def test_a_copied_cache_is_a_handle_of_its_own_tensors():
    rng = np.random.default_rng(1)
    pool = Pool(rng, [100, 40], 16, 2, 128, "e4m3")
    keep = random_tree(rng, 2, 5)
    pool.cache = copy.deepcopy(pool.cache)
    for t in (pool.k, pool.v):  # the copy does not look at what it was copied from
        t.view(torch.uint8).fill_(0x7F)
    r = run_attention(pool, 2, 5, 4, "bf16", rng, keep)
    check_all(pool, r, keep, "bf16")


@pytest.mark.parametrize("Hkv,G,d", [(1, 8191, 128), (2, 8191, 64), (2, 16383, 128)])
def test_thousands_of_query_heads_per_kv_head(Hkv, G, d):
    """128 * G rows of a KV head pass 2^32 / G: the row's token is a division that has to stay exact there.

    No prefix and no mask: row i attends tree rows 0..i.  Weights and out round to bf16 (2^-8 each); scores are fp32 sums
    of d products, (d + 8) 2^-24 sum |q||k| scale < 2^-12 for these values, and weigh twice that."""
    N, Hq = 128, Hkv * G
    gen = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, kt, vt = rnd(1, N, Hq, d), rnd(1, N, Hkv, d), rnd(1, N, Hkv, d)
    cache = E.PagedCache.allocate(1, Hkv, 16, d)
    shape = E.PagedAttnShape(B=1, N=N, Hq=Hq, max_blocks=1, max_prefix=0)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    # a margin around what the call may write, which has to stay as it is
    room = torch.full((3, N, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lroom = torch.full((3, Hq, N), 7.0, device="cuda")
    E.et_tree_attention_paged(shape, cache, i32(0)[None], i32(0), q, kt, vt, None, room[1:2], lse=lroom[1:2],
                              ws=E.new_workspace(E.et_tree_attention_paged_workspace_size(shape, cache)))
    assert all(bool((x[i] == 7).all()) for x in (room, lroom) for i in (0, 2))
    sees = torch.ones(N, N, dtype=torch.bool, device="cuda").tril()
    for g in range(Hkv):
        k, v = kt[0, :, g].float(), vt[0, :, g].float()
        for h0 in range(g * G, (g + 1) * G, 2048):
            hs = slice(h0, min(h0 + 2048, (g + 1) * G))
            z = torch.einsum("nhd,td->hnt", q[0, :, hs].float(), k) * d ** -0.5
            z = z.masked_fill(~sees, -math.inf)
            total = torch.logsumexp(z, -1)
            p = torch.exp(z - total[..., None])
            want, size = p @ v, p @ v.abs()
            got = room[1, :, hs].float().transpose(0, 1)
            err = (got - want).abs() - (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11) * size)
            assert float(err.max()) <= 0
            assert float((lroom[1, hs] - total).abs().max()) <= 2.0 ** -11


@pytest.mark.parametrize("N", [1, 17])
def test_the_longest_prefix_a_table_can_hold(N):
    """2^31 - 16 tokens, all of them in one page of 16: its softmax, and a log-sum-exp larger by ln(2^27 - 1).

    A thread's or an accumulator's sum takes up to 2^20 terms of one sign, each rounded (or cut) by 2^-23 at most: 2^-3 of
    the numerator and of the sum at the very worst.  Without the tokens the result is the tree's rows alone."""
    rng = np.random.default_rng(2)
    L = (1 << 31) - 16
    pool = Pool(rng, [16], 16, 1, 128, "e4m3")
    cols = L // 16
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((1, cols), int(pool.table[0, 0]), **i32)
    shape = E.PagedAttnShape(B=1, N=N, Hq=1, max_blocks=cols)
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, kt, vt = (torch.randn(1, N, 1, 128, generator=gen, device="cuda").bfloat16() for _ in range(3))
    out, lse = torch.zeros_like(q), torch.zeros(1, 1, N, device="cuda")
    status = torch.zeros(1, **i32)
    E.et_tree_attention_paged(shape, pool.cache, table, torch.tensor([L], **i32), q, kt, vt, None, out, lse=lse,
                              ws=E.new_workspace(E.et_tree_attention_paged_workspace_size(shape, pool.cache)),
                              dev_status=status)
    assert int(status.item()) == 0
    k, v = pool.sequence(0)
    want, wlse, size, *_ = O.paged_attention(q[0].double().cpu().numpy(), k, v, kt[0].double().cpu().numpy(),
                                             vt[0].double().cpu().numpy(), np.ones(16, bool), np.zeros((N, N), bool),
                                             128 ** -0.5)
    assert (np.abs(out[0].double().cpu().numpy() - want) <= 2.0 ** -2 * size).all()
    assert (np.abs(lse[0].double().cpu().numpy() - wlse - math.log(cols)) <= 2.0 ** -2).all()


def test_a_block_map_that_returns_almost_two_to_the_31_pages():
    """Rounds of the page loops pass 2^31 there.  The pool holds eight pages, so that the stack is cut and flagged."""
    cols, pool = (1 << 30) - 8, 8
    i32 = dict(dtype=torch.int32, device="cuda")
    room = torch.full((2 * cols + 2048,), 5, **i32)  # with a margin on both sides
    table = room[1024:-1024].view(2, cols)
    table[0, 0], table[0, 1] = 7, 6
    n, free, count = torch.full((2,), cols, **i32), torch.full((pool,), -9, **i32), torch.zeros(1, **i32)
    status = torch.zeros(1, **i32)
    shape = E.BlockMapShape(B=2, page_size=1, max_blocks=cols, num_pages=pool)
    zero = torch.zeros(2, **i32)
    E.et_block_map(shape, zero, zero, n, table, free, count, dev_status=status)
    assert int(status.item()) == E.ET_DEV_BAD_INDEX and n.tolist() == [0, 0] and count.tolist() == [pool]
    assert free.tolist() == [7, 6] + [5] * 6  # the first eight returned
    assert bool((room[:1024] == 5).all()) and bool((room[-1024:] == 5).all())
    assert int(table.min()) == int(table.max()) == -1


def test_fp32_keys_that_score_minus_infinity_leave_the_others_their_weight():
    """A warp whose first keys all score -inf (an infinite K) and whose later ones lie far below 0."""
    d, L, P = 64, 288, 32
    codes = torch.zeros(L // P, 1, P, d, dtype=torch.uint8, device="cuda")
    codes[..., 0] = 0xE0                     # e5m2: -512
    codes[0, ..., 0] = 0xFC                  # -infinity
    gen = torch.Generator(device="cuda").manual_seed(2)
    v = torch.randn(L // P, 1, P, d, generator=gen, device="cuda").to(torch.float8_e5m2)
    ones = torch.ones(L // P, 1, device="cuda")
    cache = E.PagedCache(codes.view(torch.float8_e5m2), v, ones, ones)
    q, kt, vt = (torch.zeros(1, 1, 1, d, device="cuda") for _ in range(3))
    q[..., 0], kt[..., 0] = 1.0, -512.0
    out, lse = torch.zeros_like(q), torch.zeros(1, 1, 1, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    shape = E.PagedAttnShape(B=1, N=1, Hq=1, max_blocks=L // P, dtype=E.ET_F32, scale=1.0)
    E.et_tree_attention_paged(shape, cache, i32(*range(L // P))[None], i32(L), q, kt, vt, None, out, lse=lse)
    want = v.double().view(L, d)[P:].sum(0) / (L - P + 1)  # 256 tokens and the row itself, all alike
    # equal weights: sums of 257 terms in fp32, 2^-24 a term
    assert (out.view(d).double() - want).abs().max() <= 257 * 2.0 ** -24 * v.double().abs().max()
    assert abs(float(lse) - (-512 + math.log(L - P + 1))) <= 2.0 ** -13
    # half steps of 738 (base 2: score, sum; 2^-15 each, times ln 2), of 506 (2^-16) and of the two constants (2^-25 of
    # 738 times ln 2, of 506): 1.4 * 2^-15 + 2^-16 + 1.02 * 2^-15 * 0.7 + 2^-16 < 2^-13


@pytest.mark.parametrize("L", [0, 40])
@pytest.mark.parametrize("N,d", [(1, 128), (20, 64), (20, 128)])
def test_a_query_with_an_infinity_gives_nan_and_nothing_else_does(N, d, L):
    """Also where every score of the row is -inf: the tree's keys oppose it and there is no prefix."""
    rng = np.random.default_rng(4)
    pool = Pool(rng, [L], 16, 2, d, "e4m3", cols=3)
    keep = random_tree(rng, 1, N)
    keep[0, N - 1] = N == 1  # the last of several rows attends no key of the tree
    q = torch.randn(1, N, 2, d, generator=torch.Generator().manual_seed(1)).bfloat16().float().numpy()
    clean = run_attention(pool, 1, N, 2, "bf16", np.random.default_rng(8), keep, q=q)
    hit = sorted({0, N // 2, N - 1})
    r = dict(clean, out=torch.full_like(clean["out"], 7.0), lse=torch.full_like(clean["lse"], 7.0))
    args = list(clean["args"])
    args[4], args[5], args[8] = args[4].clone(), args[5].clone(), r["out"]
    for i in hit:
        args[4][0, i, 1, 3] = math.inf
    args[5][..., 3] = -args[5][..., 3].abs() - 1  # scores of -inf
    E.et_tree_attention_paged(*args, lse=r["lse"], ws=clean["ws"], dev_status=clean["status"])
    for i in range(N):
        has_key = L > 0 or keep[0, i].any()
        for x in (r["out"][0, i, 1], r["lse"][0, 1, i]):
            assert bool(torch.isnan(x).all()) == (i in hit and has_key)
        assert not torch.isnan(r["out"][0, i, 0]).any()
        if not has_key:
            assert (r["out"][0, i] == 0).all() and torch.isneginf(r["lse"][0, :, i]).all()


@pytest.mark.parametrize("N,d", [(1, 128), (30, 64), (30, 128)])
@pytest.mark.parametrize("exp", [-104, 100])
def test_k_scales_and_queries_at_the_ends_of_their_range(N, d, exp):
    """K scales up to 2^99 on queries of 2^-104, and the other way round: plain scores."""
    rng = np.random.default_rng(9)
    pool = Pool(rng, [100], 32, 2, d, "e4m3")
    mag = np.float32(2.0) ** exp
    pool.scale[0] = (pool.scale[0] / mag).astype(np.float32)
    pool.upload()
    keep = np.zeros((1, N, N), bool)  # cached tokens only: the tree's keys have no scale
    q = torch.randn(1, N, 4, d, generator=torch.Generator().manual_seed(2)).bfloat16().float().numpy() * mag
    r = run_attention(pool, 1, N, 4, "bf16", rng, keep, q=q)
    check_all(pool, r, keep, "bf16")
