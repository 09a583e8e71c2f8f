"""Chunk attention where row_start is wrong: the sequences that are skipped, and those behind them, which keep their rows."""
import math

import pytest
import torch

from speculative_decoding_eagle_gb300 import binding as E

pytestmark = pytest.mark.gpu
DT = {"bf16": (E.ET_BF16, torch.bfloat16), "f32": (E.ET_F32, torch.float32)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_eagle_gb300 import build_lib
    build_lib.build()
    E.load()


def owners(starts, rows, max_rows):
    """The sequence of each row (-1: none) and whether any row_start is wrong, as the call's description has it."""
    own, wrong = [-1] * rows, False
    for b in range(len(starts) - 1):
        r0, r1 = starts[b], starts[b + 1]
        if r0 < 0 or r1 > rows or r1 < r0:
            wrong = True
            continue
        if r1 - r0 > max_rows:
            wrong, r1 = True, r0 + max_rows
        if any(r0 < r <= rows for r in starts[:b]):
            continue
        for r in range(r0, r1):
            assert own[r] == -1
            own[r] = b
    return own, wrong


def chain(n, width):
    """Ascending starts in which every tenth sequence is preceded by one that goes back to row 0 (it is skipped, and so is its
    successor's overlap): rows of the others are many more than their units would be counted for if all were taken."""
    s, at = [0], 0
    for b in range(n):
        at += width
        s.append(at)
        if b % 10 == 4:
            s += [0, at]
    return s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("starts,spare,max_rows", [
    ([0, 10, 0, 10, 20], 2, 64),                       # sequence 1 descends; 2 begins among 0's rows; 3 keeps its own
    ([0, 100, 0, 100, 0, 100, 0, 100, 120], 0, 128),   # the same rows named four times
    ([0, 300, 0, 300, 0, 300, 301, 302, 303, 600], 5, 300),
    ([0, 40, 1000, 40, 70], 0, 64),                    # out of range: two are skipped, no more
    ([5, -3, 9, 9, 12], 4, 64),
    ([0, 8, 8, 3, 8, 30], 1, 10),                      # descends, and a last one that is cut
    (chain(60, 7), 3, 9),                              # past the batches that are ordered
    (chain(700, 1), 0, 2),                             # more sequences than a block has threads
    (list(range(1100)) + [50, 60, 1099, 1105], 2, 64),  # right for two rounds of threads, then back into their rows
    ([0, 1500] + list(range(0, 1400, 2)) + [1500, 1510], 0, 1500),  # a first sequence that has everyone's rows but the last's
])
def test_wrong_starts(starts, spare, max_rows, dtype):
    et, dt = DT[dtype]
    Hq, Hkv, d, P, L, cols = 4, 2, 64, 32, 70, 3
    B, rows = len(starts) - 1, max(s for s in starts if s < 1000) + spare
    g = torch.Generator(device="cuda").manual_seed(rows + B)
    cache = E.PagedCache.allocate(cols, Hkv, P, d)
    for pages, scale in ((cache.k_pages, cache.k_scale), (cache.v_pages, cache.v_scale)):
        x = torch.randn(cols, Hkv, P, d, generator=g, device="cuda")
        pages.view(torch.uint8).copy_((x * 64).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        scale.fill_(2.0 ** -6)
    table = torch.arange(cols, dtype=torch.int32, device="cuda").repeat(B, 1)  # one prefix for all
    q, k, v = (torch.randn(rows, h, d, generator=g, device="cuda").to(dt) for h in (Hq, Hkv, Hkv))
    out, lse = torch.full((rows, Hq, d), 7.0, dtype=dt, device="cuda"), torch.full((rows, Hq), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    shape = E.ChunkAttnShape(B=B, rows=rows, Hq=Hq, max_rows=max_rows, max_blocks=cols, dtype=et)
    ws = E.new_workspace(E.et_chunk_attention_paged_workspace_size(shape, cache))
    E.et_chunk_attention_paged(shape, cache, table, torch.full((B,), L, dtype=torch.int32, device="cuda"),
                               torch.tensor(starts, dtype=torch.int32, device="cuda"), q, k, v, out, lse=lse, ws=ws, dev_status=status)
    torch.cuda.synchronize()
    own, wrong = owners(starts, rows, max_rows)
    assert wrong and int(status.item()) == E.ET_DEV_BAD_INDEX
    held = lambda x, s: (x.float() * s[:, :, None, None]).transpose(0, 1).reshape(Hkv, -1, d)[:, :L].double()  # noqa: E731
    kp, vp = held(cache.k_pages, cache.k_scale), held(cache.v_pages, cache.v_scale)
    own = torch.tensor(own, device="cuda")
    r = torch.arange(rows, device="cuda")
    sees = (own[:, None] == own[None]) & (r[None] <= r[:, None])
    sees = torch.cat([torch.ones(rows, L, dtype=torch.bool, device="cuda"), sees], 1)
    for h in range(Hq):
        kk, vv = (torch.cat([p[h // 2], n[:, h // 2].double()]) for p, n in ((kp, k), (vp, v)))
        z = (q[:, h].double() @ kk.T / math.sqrt(d)).masked_fill(~sees, -math.inf)
        total = torch.logsumexp(z, 1)
        p = torch.exp(z - total[:, None])
        want, mass = p @ vv, p @ vv.abs()
        # fp32: sums of a few hundred terms (2^-24 each) and exponentials.  bf16: weights and outputs rounded by 2^-8 at most
        tol = 2e-5 * want.abs().amax(1, keepdim=True) if dtype == "f32" else 2.0 ** -8 * (want.abs() + mass)
        live = own >= 0
        assert bool(((out[:, h].double() - want).abs() <= tol)[live].all())
        assert bool(((lse[:, h].double() - total).abs() <= 1e-5 * (1 + total.abs()))[live].all())
        assert bool((out[~live] == 7).all()) and bool((lse[~live] == 7).all())
