"""Rotation, chunk attention and sampling without a GPU: frequencies against their definitions, and every argument that the
calls refuse (before any launch, so that none is needed)."""
import copy
import ctypes
import math
import pickle

import numpy as np
import pytest
import torch

from speculative_decoding_eagle_gb300 import binding as E
from speculative_decoding_eagle_gb300 import build_lib

FAKE = 0x100000  # a non-null, 256-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return E.load()


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------
def test_plain_linear_and_base_frequencies(lib):
    n, theta = 32, 10000.0
    base = np.array([theta ** (-i / n) for i in range(n)])
    f, factor = E.et_rotary_frequencies(64)
    np.testing.assert_allclose(f.numpy(), base, rtol=4e-16)
    assert factor == 1.0 and f[0] == 1.0
    f, factor = E.et_rotary_frequencies(64, theta, E.ET_ROPE_LINEAR, 4.0)
    np.testing.assert_allclose(f.numpy(), base / 4, rtol=4e-16)
    f, _ = E.et_rotary_frequencies(64, theta, E.ET_ROPE_BASE, 4.0)
    # the slowest pair is slowed down `scale` times, the fastest not at all
    assert f[0] == 1.0 and abs(f[-1] / base[-1] - 0.25) < 1e-12


def test_ramp_and_band_frequencies(lib):
    n, theta, scale, trained = 64, 10000.0, 8.0, 4096.0
    base = np.array([theta ** (-i / n) for i in range(n)])
    turns = trained * base / (2 * math.pi)
    f, factor = E.et_rotary_frequencies(128, theta, E.ET_ROPE_RAMP, scale, trained, 32.0, 1.0)
    r = f.numpy() / base
    assert abs(factor - (0.1 * math.log(8) + 1)) < 1e-7
    assert np.all(np.diff(r) <= 1e-15) and r[0] == 1.0 and abs(r[-1] - 1 / 8) < 1e-15
    lo = math.floor(n * math.log(trained / (32 * 2 * math.pi)) / math.log(theta))
    hi = math.ceil(n * math.log(trained / (2 * math.pi)) / math.log(theta))
    want = [1 - min(max((i - lo) / (hi - lo), 0), 1) for i in range(n)]
    np.testing.assert_allclose(r, [k + (1 - k) / 8 for k in want], rtol=1e-14)
    f, factor = E.et_rotary_frequencies(128, theta, E.ET_ROPE_BANDS, scale, trained, 4.0, 1.0)
    r = f.numpy() / base
    assert factor == 1.0
    np.testing.assert_array_equal(r[turns >= 4], 1.0)
    np.testing.assert_allclose(r[turns <= 1], 1 / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 4)
    k = (turns[mid] - 1) / 3
    np.testing.assert_allclose(r[mid], k + (1 - k) / 8, rtol=1e-14)


@pytest.mark.parametrize("bad", [dict(rot=0), dict(rot=3), dict(rot=-2), dict(rot=514), dict(theta=1.0), dict(theta=math.nan),
                                 dict(theta=math.inf), dict(scaling=5), dict(scaling=-1), dict(scaling=1, scale=0.5),
                                 dict(scaling=2, scale=math.nan), dict(scaling=2, scale=2.0, rot=2), dict(scaling=3, trained=0.0),
                                 dict(scaling=3, fast=1.0, slow=1.0), dict(scaling=4, slow=0.0), dict(scaling=4, fast=math.inf)])
def test_frequencies_refused(lib, bad):
    a = dict(rot=64, theta=10000.0, scaling=0, scale=2.0, trained=4096.0, fast=4.0, slow=1.0)
    a.update(bad)
    with pytest.raises(E.EtError) as e:
        E.et_rotary_frequencies(**a)
    assert e.value.status == E.ET_ERR_INVALID_ARG


# ---------------------------------------------------------------------------
# refusals of the C calls
# ---------------------------------------------------------------------------
def rotary_status(lib, positions=FAKE, freq=FAKE, q=FAKE, k=FAKE, qo=2 * FAKE, ko=2 * FAKE, **over):
    a = dict(rows=4, Hq=4, Hkv=2, d=64, rot=64, layout=0, dtype=0, factor=1.0, q_stride=256, k_stride=128, q_out_stride=256,
             k_out_stride=128)
    a.update(over)
    s = E.RotaryShapeC(*(a[n] for n, _ in E.RotaryShapeC._fields_))
    return lib.et_rotary(ctypes.byref(s), positions, freq, q, k, qo, ko, None)


@pytest.mark.parametrize("over,want", [
    (dict(positions=None), 1), (dict(freq=None), 1), (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(ko=None), 1),
    (dict(k=None, ko=None), 1), (dict(Hkv=0), 1), (dict(rows=0), 1), (dict(Hq=0), 1), (dict(d=60), 1), (dict(d=0), 1),
    (dict(rot=8), 1), (dict(rot=72), 1), (dict(rot=24), 1), (dict(rot=0), 1), (dict(factor=math.inf), 1),
    (dict(factor=math.nan), 1), (dict(layout=2), 1), (dict(dtype=2), 1), (dict(q_stride=255), 1), (dict(q_stride=252), 1),
    (dict(k_stride=127), 1), (dict(q_out_stride=0), 1), (dict(k_out_stride=-8), 1), (dict(q_stride=260), 1),
    (dict(q=FAKE + 8), 1), (dict(ko=FAKE + 2), 1), (dict(positions=FAKE + 2), 1), (dict(freq=FAKE + 4), 1),
    (dict(qo=FAKE, q_out_stride=512), 1), (dict(ko=FAKE, k_out_stride=256), 1), (dict(d=520, q_stride=4096, k_stride=4096, q_out_stride=4096, k_out_stride=4096), 2)])
def test_rotary_refuses(lib, over, want):
    assert rotary_status(lib, **over) == want


def cache(Hkv=2, d=128, page_size=64, fmt=0, num_pages=10, stride=2 * 64 * 128, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE):
    return E.PagedCacheC(Hkv, d, page_size, fmt, num_pages, stride, k, v, ks, vs)


def chunk_args(**over):
    a = dict(B=2, Hq=4, rows=100, max_rows=60, max_blocks=8, dtype=0, scale=0.1, max_prefix=512, num_splits=0, q_stride=512,
             k_stride=256, v_stride=256)
    a.update(over)
    return E.ChunkAttnShapeC(*(a[n] for n, _ in E.ChunkAttnShapeC._fields_))


def chunk_status(lib, cache_=None, table=FAKE, plen=FAKE, start=FAKE, q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=None, ws=FAKE,
                 ws_bytes=1 << 40, **over):
    c = cache_ or cache()
    return lib.et_chunk_attention_paged(ctypes.byref(chunk_args(**over)), ctypes.byref(c), table, plen, start, q, k, v, out,
                                        lse, None, ws, ws_bytes, None)


@pytest.mark.parametrize("over,want", [
    (dict(table=None), 1), (dict(plen=None), 1), (dict(start=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(out=None), 1), (dict(B=0), 1), (dict(rows=0), 1), (dict(max_rows=0), 1), (dict(max_rows=-5), 1), (dict(Hq=0), 1),
    (dict(Hq=3), 1), (dict(max_blocks=0), 1), (dict(max_prefix=-1), 1), (dict(num_splits=-1), 1), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(dtype=2), 1), (dict(q_stride=511), 1),
    (dict(q_stride=516), 1), (dict(k_stride=128), 1), (dict(v_stride=260), 1), (dict(v_stride=1 << 40), 1), (dict(q=FAKE + 8), 1),
    (dict(v=FAKE + 2), 1), (dict(out=FAKE + 4), 1), (dict(start=FAKE + 1), 1), (dict(lse=FAKE + 2), 1), (dict(B=70000), 2),
    (dict(max_blocks=1 << 26), 2), (dict(num_splits=3, ws=None), 3), (dict(num_splits=3, ws_bytes=100), 3),
    (dict(num_splits=3, ws=FAKE + 16), 3)])
def test_chunk_attention_refuses(lib, over, want):
    assert chunk_status(lib, **over) == want


@pytest.mark.parametrize("bad,want", [(dict(Hkv=0), 1), (dict(d=96), 2), (dict(page_size=24), 2), (dict(page_size=272), 2),
                                      (dict(fmt=2), 1), (dict(num_pages=0), 1), (dict(stride=100), 1), (dict(k=None), 1),
                                      (dict(v=FAKE + 8), 1), (dict(ks=None), 1)])
def test_chunk_attention_refuses_caches(lib, bad, want):
    assert chunk_status(lib, cache_=cache(**bad)) == want
    c = cache(**bad)
    assert lib.et_chunk_attention_paged_splits(ctypes.byref(chunk_args()), ctypes.byref(c)) == -1 or bad.keys() & {"k", "v", "ks"}


def test_chunk_attention_plans(lib):
    def plan(**over):
        s, c = chunk_args(**over), cache()
        return (lib.et_chunk_attention_paged_splits(ctypes.byref(s), ctypes.byref(c)),
                lib.et_chunk_attention_paged_workspace_size(ctypes.byref(s), ctypes.byref(c)))
    assert plan(dtype=1) == (1, 0)                                        # fp32: one part
    assert plan(num_splits=1) == (1, 0)
    assert plan(max_rows=2 ** 31 - 1) == plan(max_rows=100)                # a bound past the rows is the rows
    S, ws = plan(num_splits=3)
    # (tiles of 256 rows: 100 * 2 / 256 of them whole, and one that each sequence ends in) x heads x parts x 256 rows
    assert S == 3 and ws == 16384 * 4 + (0 + 2) * 2 * 3 * 256 * (8 + 128 * 4)
    assert plan(num_splits=500)[0] == 5                                   # no more parts than tiles of 128 keys: 4 + 1
    assert plan(B=1, rows=1, max_rows=1, max_prefix=10 ** 9, max_blocks=4096)[0] > 4   # few rows, many keys
    assert plan(B=64, rows=60000, max_rows=60000, num_splits=0)[0] == 1   # many rows
    assert plan(B=4000, rows=10 ** 6, max_rows=10 ** 6, num_splits=4) == (1, 0)        # more tiles than counters


def sample_status(lib, logits=FAKE, T=None, k=None, p=None, m=None, u=FAKE, tok=FAKE, lp=None, tr=None, **over):
    a = dict(B=2, V=100, row_stride=100, out_stride=0)
    a.update(over)
    s = E.SampleShapeC(*(a[n] for n, _ in E.SampleShapeC._fields_))
    return lib.et_sample(ctypes.byref(s), logits, T, k, p, m, u, tok, lp, tr, None, None)


@pytest.mark.parametrize("over,want", [
    (dict(logits=None), 1), (dict(u=None), 1), (dict(tok=None), 1), (dict(B=0), 1), (dict(V=0), 1), (dict(row_stride=99), 1),
    (dict(tr=FAKE), 1), (dict(tr=FAKE, out_stride=99), 1), (dict(logits=FAKE + 2), 1), (dict(T=FAKE + 1), 1), (dict(k=FAKE + 2), 1),
    (dict(p=FAKE + 3), 1), (dict(m=FAKE + 1), 1), (dict(tok=FAKE + 2), 1), (dict(lp=FAKE + 1), 1), (dict(V=262145, row_stride=262145), 2),
    (dict(B=1 << 25), 2)])
def test_sample_refuses(lib, over, want):
    assert sample_status(lib, **over) == want


def test_null_shapes_are_refused(lib):
    assert lib.et_rotary(None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == 1
    assert lib.et_sample(None, FAKE, None, None, None, None, FAKE, FAKE, None, None, None, None) == 1
    assert lib.et_chunk_attention_paged(None, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, 0, None) == 1
    assert lib.et_rotary_frequencies(None, None, None) == 1


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def test_the_binding_takes_cuda_tensors_only(lib):
    z = torch.zeros(2, 10)
    with pytest.raises(ValueError):
        E.et_sample(z, torch.zeros(2), torch.zeros(2, dtype=torch.int32))
    q = torch.zeros(2, 1, 64)
    with pytest.raises(ValueError):
        E.et_rotary(E.RotaryShape(rows=2, Hq=1, d=64, dtype=E.ET_F32), torch.zeros(2, dtype=torch.int32),
                    torch.zeros(32, dtype=torch.float64), q, q)
    with pytest.raises(ValueError):
        E.et_rotary(E.RotaryShape(rows=2, Hq=1, d=64, Hkv=1), torch.zeros(2, dtype=torch.int32),
                    torch.zeros(32, dtype=torch.float64), q, q)


def test_shapes_can_be_copied_and_pickled():
    for s in (E.ChunkAttnShape(B=1, rows=4, Hq=2, max_rows=4, max_blocks=3), E.RotaryShape(rows=3, Hq=1, d=64)):
        if isinstance(s, E.RotaryShape):
            s.with_strides((64, 0, 64, 0))
        for t in (copy.copy(s), copy.deepcopy(s), pickle.loads(pickle.dumps(s))):
            assert t == s
