"""Chunk attention over long prefixes: many keys that are each far too small for the sum, and together are not (fp32), and the
tensor cores' sums in parts (bf16)."""
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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("first,log2_below", [(True, 26.0), (False, 26.0), (True, 31.0)])
def test_many_small_weights_count(first, log2_below, d):
    """2^18 keys of weight 2^-26 (2^-31) beside one of weight 1: their mass is 2^-8 (2^-13) of it."""
    L, P = 1 << 18, 256
    x = Batch([L], [5], 2, 1, d, P, dtype="f32", seed=30)
    for pages, scale in ((x.cache.k_pages, x.cache.k_scale), (x.cache.v_pages, x.cache.v_scale)):
        pages.view(torch.uint8).zero_()
        scale.fill_(1.0)
    one, two = (torch.tensor(v).to(torch.float8_e4m3fn).view(torch.uint8).item() for v in (1.0, 2.0))
    at = 0 if first else L - 1
    page, slot = int(x.table[0, at // P]), at % P
    x.cache.k_pages.view(torch.uint8)[page, 0, slot, 0] = one
    x.cache.v_pages.view(torch.uint8).fill_(two)
    x.cache.v_pages.view(torch.uint8)[page, 0, slot] = one
    x.q.zero_()
    x.q[:, :, 0] = log2_below * math.log(2) * math.sqrt(d)
    x.k.zero_()                                       # the new rows weigh as little as the others
    x.v.fill_(2.0)
    x.run()
    assert int(x.status.item()) == 0
    out, lse, _ = x.exact()
    # A score near 22 is off by 2^-23 of it, 3e-6.  Each value goes through at most 512 sums inside a group of tiles and 513
    # of groups, off by half a step, 2^-25 of what they hold, each: 1025 * 2^-25 = 3.1e-5, as the sum of weights is
    tol = 2 * 1025 * 2.0 ** -25 + 6e-6
    assert bool(((x.out[:5].double() - out[:5]).abs() <= tol * out[:5].abs()).all())
    assert bool(((x.lse[:5].double() - lse[:5]).abs() <= tol + 2.0 ** -22 * lse[:5].abs()).all())
    # without the small keys the output would be 1
    assert bool((out[:5] > 1 + 0.9 * 2.0 ** (18 - log2_below)).all())


@pytest.mark.parametrize("rows", [1, 300])
def test_long_sums_of_the_tensor_cores_in_parts(rows):
    """2^22 keys with values between 1 and 2 (in one part the sums would lose 1.6%): parts of 2^18 keys keep them."""
    L, P, d = 1 << 22, 256, 64
    cols = L // P
    g = torch.Generator(device="cuda").manual_seed(31)
    cache = E.PagedCache.allocate(cols, 1, P, d)
    for pages, x in ((cache.k_pages, torch.randn(cols, 1, P, d, generator=g, device="cuda")),
                     (cache.v_pages, 1 + torch.rand(cols, 1, P, d, generator=g, device="cuda"))):
        pages.view(torch.uint8).copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    q, k, v = (torch.randn(rows, 1, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    v = v.abs() + 1
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = torch.full((rows, 1, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((rows, 1), 7.0, device="cuda")
    st = i32(0)
    shape = E.ChunkAttnShape(B=1, rows=rows, Hq=1, max_rows=rows, max_blocks=cols, num_splits=17)
    ws = E.new_workspace(E.et_chunk_attention_paged_workspace_size(shape, cache))
    E.et_chunk_attention_paged(shape, cache, torch.arange(cols, device="cuda", dtype=torch.int32)[None], i32(L), i32(0, rows), q, k, v,
                               out, lse=lse, ws=ws, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for r in {0, rows // 2, rows - 1}:
        keys = torch.cat([cache.k_pages.float().reshape(L, d), k[:r + 1, 0].float()])
        z = keys.double() @ q[r, 0].double() / 8
        p = torch.softmax(z, 0)
        want = p @ torch.cat([cache.v_pages.float().reshape(L, d), v[:r + 1, 0].float()]).double()
        # the output's rounding (2^-8), the weights' (2^-11; the new rows' few count as little as they weigh), and the sums':
        # 2^-27 a key of a part, 2^18 of them
        assert bool(((out[r, 0].double() / want - 1).abs() <= 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -9).all())
        assert abs(float(lse[r, 0]) - float(torch.logsumexp(z, 0))) <= 1e-5 * (1 + abs(float(lse[r, 0])))
