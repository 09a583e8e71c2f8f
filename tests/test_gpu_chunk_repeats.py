"""Chunk attention called again on the same workspace: everything is written anew, statuses stay clean, and the bits are the
same."""
import math

import pytest
import torch

from speculative_decoding_eagle_gb300 import binding as E
from test_gpu_chunk import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_eagle_gb300 import build_lib
    build_lib.build()


def again(x, **kw):
    """A call after which every row of a sequence has been written (no sum of these inputs is 7 to the last bit)."""
    x.out.fill_(7.0)
    x.lse.fill_(7.0)
    x.status.zero_()
    ws = x.run(**kw)
    assert int(x.status.item()) == 0
    held = torch.zeros(x.T, dtype=torch.bool, device="cuda")
    for b, n in enumerate(x.prefix):
        if n >= 0:
            held[int(x.start[b]):int(x.start[b + 1])] = True
    assert bool((x.lse[held] != 7).all()) and bool((x.out[held] != 7).any(-1).all())
    assert bool((x.lse[~held] == 7).all()) and bool((x.out[~held] == 7).all())
    return ws


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("splits", [0, 1, 2, 5])
@pytest.mark.parametrize("prefix,rows,Hq,Hkv,P,d", [
    ([2100], [300], 2, 2, 64, 128),
    ([3000], [17], 2, 1, 32, 64),
    ([700, 0, 1500, -1], [300, 500, 1, 9], 4, 2, 128, 128),
    ([0], [700], 1, 1, 64, 64),
    ([500] * 40, [1] * 39 + [90], 4, 4, 16, 128),   # past the batches that are ordered
])
def test_the_same_bits_into_cleared_outputs(prefix, rows, Hq, Hkv, P, d, splits, dtype):
    x = Batch(prefix, rows, Hq, Hkv, d, P, dtype=dtype, seed=20 + splits)
    ws = again(x, splits=splits)
    x.check()
    first = x.out.clone(), x.lse.clone()
    for _ in range(5):
        again(x, splits=splits, ws=ws)
        assert torch.equal(first[0], x.out) and torch.equal(first[1], x.lse)


def test_the_same_bits_in_a_last_round_of_parts():
    x = Batch([2000], [700], 64, 8, 128, 64, seed=21)
    ws = again(x)
    x.check()
    first = x.out.clone(), x.lse.clone()
    for _ in range(5):
        again(x, ws=ws)
        assert torch.equal(first[0], x.out) and torch.equal(first[1], x.lse)


@pytest.mark.parametrize("splits", [1, 4, 9])
def test_scores_far_apart_in_parts(splits):
    """Scores of thousands, whose maximum moves from tile to tile and from part to part."""
    x = Batch([1024], [130], 1, 1, 128, 64, seed=22)
    ramp = 2.0 ** (torch.arange(16, device="cuda") / 2)
    x.cache.k_scale[x.table[0].long()] = (ramp * 2.0 ** -8)[:, None]
    x.q[::2] *= 30
    again(x, splits=splits)
    out, lse, mass = x.exact()
    pages = x.table[0].long()
    keys = (x.cache.k_pages.float()[pages, 0] * x.cache.k_scale[pages, 0, None, None]).reshape(-1, 128).double()
    # A score is a sum of 128 products in fp32, off by at most 128 * 2^-23 of the sum of their magnitudes, A; a weight and
    # the log-sum-exp move by as much.  Then the weights' and the output's roundings, 2^-8 at most each
    A = (x.q[:130, 0].double().abs() @ keys.abs().T).amax(1) / math.sqrt(128)
    A = torch.maximum(A, (x.q[:130, 0].double().abs() @ x.k[:130, 0].double().abs().T).amax(1) / math.sqrt(128))
    slack = 2.0 ** -16 * A
    assert bool(((x.lse[:130, 0].double() - lse[:130, 0]).abs() <= slack + 1e-5 * (1 + lse[:130, 0].abs())).all())
    tol = (2.0 ** -8 + 2 * torch.expm1(slack)[:, None]) * (out[:130, 0].abs() + mass[:130, 0])
    assert bool(((x.out[:130, 0].double() - out[:130, 0]).abs() <= tol).all())


def test_two_calls_at_once():
    """Two streams, each with a workspace of its own, give what the calls give alone."""
    calls = [(Batch([2100, 0], [300, 90], 4, 2, 128, 64, seed=23), 3), (Batch([1500] * 6, [1] * 6, 8, 2, 64, 16, seed=24), 2),
             (Batch([400], [700], 2, 2, 128, 32, seed=25), 0)]
    want, spaces = [], []
    for x, splits in calls:
        spaces.append(again(x, splits=splits))
        x.check()
        want.append((x.out.clone(), x.lse.clone()))
        x.out.fill_(7.0)
        x.lse.fill_(7.0)
    streams = [torch.cuda.Stream() for _ in calls]
    shapes = [E.ChunkAttnShape(B=len(x.prefix), rows=x.T, Hq=x.Hq, max_rows=max(x.rows), max_blocks=x.table.shape[1],
                               num_splits=splits) for x, splits in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for (x, _), ws, s, shape in zip(calls, spaces, streams, shapes):
            E.et_chunk_attention_paged(shape, x.cache, x.table, x.plen, x.start, x.q, x.k, x.v, x.out, lse=x.lse, ws=ws,
                                       dev_status=x.status, stream=s)
    torch.cuda.synchronize()
    for (x, _), (out, lse) in zip(calls, want):
        assert int(x.status.item()) == 0 and torch.equal(out, x.out) and torch.equal(lse, x.lse)
