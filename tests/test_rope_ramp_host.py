"""The ramp of et_rotary_frequencies where a model was trained on so many tokens that its slowest pairs turn more often than
`slow` times: the ramp ends past the last pair then, and that pair keeps part of its frequency."""
import math

import numpy as np
import pytest

from speculative_decoding_eagle_gb300 import binding as E
from speculative_decoding_eagle_gb300 import build_lib


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    E.load()


def kept(rot, theta, trained, fast, slow):
    """Share of the unscaled frequency of each pair: 1 at the dim that turns `fast` times and before, 0 from the one that turns
    `slow` times on, both ends rounded outward to whole pairs and held within 0 .. rot - 1."""
    n = rot // 2
    dim = lambda turns: n * math.log(trained / (turns * 2 * math.pi)) / math.log(theta)  # noqa: E731
    lo, hi = max(0, math.floor(dim(fast))), min(rot - 1, math.ceil(dim(slow)))
    return np.array([1 - min(max((i - lo) / max(hi - lo, 1e-3), 0), 1) for i in range(n)])


@pytest.mark.parametrize("rot,theta,scale,trained", [
    (128, 1e4, 8.0, 131072.0),     # the last pair turns 2.4 times
    (128, 1e4, 8.0, 65536.0),      # 1.2 times
    (64, 1e6, 4.0, 8388608.0),
    (32, 1e4, 2.0, 10.0 ** 6),
    (16, 100.0, 16.0, 10.0 ** 7),  # every pair turns more than 32 times
    (128, 1e4, 8.0, 4096.0),       # the ramp ends among the pairs
    (128, 5e5, 32.0, 8192.0),
])
def test_the_ramp_ends_where_a_pair_turns_slow_times(rot, theta, scale, trained):
    n = rot // 2
    base = np.array([theta ** (-i / n) for i in range(n)])
    turns = trained * base / (2 * math.pi)
    f, _ = E.et_rotary_frequencies(rot, theta, E.ET_ROPE_RAMP, scale, trained, 32.0, 1.0)
    share = f.numpy() / base
    keep = kept(rot, theta, trained, 32.0, 1.0)
    # powers, logarithms and quotients of doubles: a few units of 2^-53 each, and the power's exponent of up to 14 nats
    np.testing.assert_allclose(share, keep + (1 - keep) / scale, rtol=1e-13)
    # a pair that turns more than `slow` times is not slowed down all the way, whichever pair it is
    assert np.all(share[turns > 1.001] > 1 / scale)
