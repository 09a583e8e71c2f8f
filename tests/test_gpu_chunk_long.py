"""fp32 chunk attention over long prefixes: many keys that are each far too small for the sum, and together are not."""
import math

import pytest
import torch

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
