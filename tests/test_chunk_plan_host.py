"""How many parts chunk attention takes over prefixes of more than 2^18 keys."""
import ctypes

import pytest

from speculative_decoding_eagle_gb300 import binding as E
from speculative_decoding_eagle_gb300 import build_lib

FAKE = 0x100000  # a non-null, 256-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return E.load()


def plan(lib, max_prefix, rows=60000, splits=0, dtype=0, Hkv=2):
    c = E.PagedCacheC(Hkv, 128, 256, 0, 1000, Hkv * 256 * 128, FAKE, FAKE, FAKE, FAKE)
    s = E.ChunkAttnShapeC(1, 2 * Hkv, rows, rows, (1 << 23) - 1, dtype, 0.1, max_prefix, splits, 256 * Hkv, 128 * Hkv, 128 * Hkv)
    return (lib.et_chunk_attention_paged_splits(ctypes.byref(s), ctypes.byref(c)),
            lib.et_chunk_attention_paged_workspace_size(ctypes.byref(s), ctypes.byref(c)))


def test_a_part_has_at_most_2_18_keys(lib):
    rows = 60000                                           # 469 tiles of new rows, more units than SMs
    units = 2 * ((2 * rows + 255) // 256)
    for prefix in ((1 << 19), (1 << 20) + 77, 1 << 22, 1 << 24):
        tiles = -(-prefix // 128) + -(-rows // 128)
        S, ws = plan(lib, prefix)
        assert S == min(64, -(-tiles // 2048)) > 1
        assert ws == 16384 * 4 + units * S * 256 * (8 + 4 * 128)
    assert plan(lib, (1 << 31) - 256)[0] == 64             # no more parts than that
    assert plan(lib, 1 << 22, splits=1) == (1, 0)          # as asked for
    assert plan(lib, 1 << 22, dtype=1) == (1, 0)
    assert plan(lib, 1 << 22, rows=1)[0] >= 16             # few rows have more parts anyway
