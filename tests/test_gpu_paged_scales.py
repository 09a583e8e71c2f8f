"""The paged attention on caches as the library's own commit writes them, whatever the size of V.

A page's V scale is about its largest magnitude / the format's largest value,
so it shrinks with V and with the format's range.  Cached and tree keys have
to be weighed on one footing: the result may not depend on how large V is,
nor on which of the two kinds of key a row attends most.
"""
import numpy as np
import pytest
import torch

import oracle as O
from speculative_decoding_eagle_gb300 import binding as E
from tests.test_gpu_paged import F8, check_attention, dev, mask_words, random_tree

pytestmark = pytest.mark.gpu


def quantised(x, fmt, P):
    """Rows [L, Hkv, d] as pages: codes [pages, Hkv, P, d] and scales [pages, Hkv], as et_kv_commit_paged makes them."""
    L, Hkv, d = x.shape
    pages = -(-L // P)
    codes, scale = np.zeros((pages, Hkv, P, d), np.uint8), np.zeros((pages, Hkv), np.float32)
    for p in range(pages):
        rows = x[p * P:(p + 1) * P]
        for g in range(Hkv):
            s = O.page_scale(np.abs(rows[:, g]).max(), fmt)
            codes[p, g, :len(rows)] = O.encode(rows[:, g] / s, fmt)
            scale[p, g] = s
    return codes, scale


def peaked(fmt, d, N, v_size, splits, lens=(1500, 333), Hkv=2, P=48, nats=7.0, dtype=torch.bfloat16, tree_v=1.0,
           lone=()):
    """Rows whose own key scores `nats` above the cached ones, V of mean half its deviation, sizes v_size * N(0, 1).
    Rows `lone` are attended by themselves alone, and their V is 2^60 times as large."""
    rng = np.random.default_rng(int(d + N + splits))
    B, scale = len(lens), d ** -0.5
    bf = lambda x: torch.from_numpy(x.astype(np.float32)).bfloat16().float().numpy()  # noqa: E731
    q = bf(rng.standard_normal((B, N, Hkv, d)))
    # the own score nats, those of other rows' keys about N(0, 0.1); cached scores about N(0, 0.1) too
    kt = bf(0.1 * rng.standard_normal((B, N, Hkv, d)) + q * (nats / scale / (q ** 2).sum(-1, keepdims=True)))
    vt = bf((rng.standard_normal((B, N, Hkv, d)) + 0.5) * v_size * tree_v)
    codes, scales, tables, kc, vc, at = [[], []], [[], []], [], [], [], 0
    cols = max(-(-n // P) for n in lens)
    for n in lens:
        k, v = 0.1 * rng.standard_normal((n, Hkv, d)), (rng.standard_normal((n, Hkv, d)) + 0.5) * v_size
        for x, (y, store) in enumerate(((k, kc), (v, vc))):
            c, s = quantised(y, fmt, P)
            codes[x].append(c)
            scales[x].append(s)
            store.append(O.dequantised(c, s, fmt, np.arange(len(c)), n))
        tables.append(np.concatenate([np.arange(len(c)) + at, np.full(cols - len(c), -1)]))
        at += len(c)
    pages = [dev(np.concatenate(c)).view(F8[fmt]) for c in codes]
    cache = E.PagedCache(pages[0], pages[1], *[dev(np.concatenate(s)) for s in scales])
    keep = random_tree(rng, B, N)
    for j in lone:
        keep[:, :, j] = False
        keep[:, j, j] = True
        vt[:, j] *= np.float32(2.0 ** 60)
    shape = E.PagedAttnShape(B=B, N=N, Hq=Hkv, max_blocks=cols, max_prefix=max(lens), num_splits=splits,
                             dtype=E.ET_BF16 if dtype == torch.bfloat16 else E.ET_F32)
    ws = E.new_workspace(E.et_tree_attention_paged_workspace_size(shape, cache))
    out, lse = torch.zeros(B, N, Hkv, d, dtype=dtype, device="cuda"), torch.zeros(B, Hkv, N, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.et_tree_attention_paged(shape, cache, dev(np.stack(tables).astype(np.int32)), dev(np.array(lens, np.int32)),
                              dev(q).to(dtype), dev(kt).to(dtype), dev(vt).to(dtype), dev(mask_words(keep).view(np.int64)),
                              out, lse=lse, ws=ws, dev_status=status)
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert int(status.item()) == 0
    for b, n in enumerate(lens):
        ref = O.paged_attention(q[b], kc[b], vc[b], kt[b], vt[b], np.ones(n, bool), keep[b], scale)
        yield got[b], glse[b], ref, n


# Weights round to fp16 within 2^-11 of their value down to fp16's smallest normal value, 2^-14.  A row's reference
# leaves its largest key 2^3 at least; here a cached key lies below the largest by 7 nats and 1.3 nats of spread (2^-12),
# and by the page scales' ratio (powers of two of largest magnitudes of like data: 2^-2): 2^-11, so the bound of
# check_attention, relative to each weight, holds.
@pytest.mark.parametrize("v_size", [2.0 ** -20, 2.0 ** -10, 0.05, 1.0, 2.0 ** 10])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("d,N,splits", [(64, 1, 1), (64, 40, 2), (128, 1, 1), (128, 1, 3), (128, 61, 1), (128, 61, 3),
                                        (128, 128, 1)])
def test_a_key_of_the_tree_far_above_the_cached_ones(d, N, splits, fmt, v_size):
    for got, glse, ref, n in peaked(fmt, d, N, v_size, splits):
        check_attention(got, glse, ref, d, "bf16", n, N)


@pytest.mark.parametrize("d,N", [(64, 1), (128, 1), (128, 61)])
@pytest.mark.parametrize("tree_v", [0.0, 2.0 ** -30, 2.0 ** 4])
def test_a_tree_whose_v_is_of_another_size(d, N, tree_v):
    """V of the tree zero, tiny or 16 times the cache's: 4 nats and 2^4 put a cached weight at 2^-11 once more."""
    for got, glse, ref, n in peaked("e4m3", d, N, 1.0, 2, nats=4.0, tree_v=tree_v):
        check_attention(got, glse, ref, d, "bf16", n, N)


def test_fp32_takes_v_of_any_size():
    for v_size in (2.0 ** -20, 1.0, 2.0 ** 10):
        for got, glse, ref, n in peaked("e5m2", 64, 5, v_size, 0, lens=(200, 33), dtype=torch.float32):
            check_attention(got, glse, ref, 64, "f32", n, 5)


@pytest.mark.parametrize("d,N,splits", [(64, 40, 1), (128, 2, 1), (128, 16, 3), (128, 61, 1), (128, 128, 2)])
def test_a_row_of_the_tree_does_not_decide_about_rows_that_do_not_attend_it(d, N, splits):
    """Padding of a tree may hold anything finite: rows beside it get what they get without it."""
    for got, glse, ref, n in peaked("e4m3", d, N, 0.05, splits, nats=5.0, lone=(N // 2, N - 1)):
        check_attention(got, glse, ref, d, "bf16", n, N)
