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
