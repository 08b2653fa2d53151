"""Reading windows of the 8-bit cache that begin anywhere a 32-bit number can say (needs a
GPU): what lies before a sequence or past its end is zeros."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv_harness import cache_of, pools, read_all

pytestmark = pytest.mark.gpu


def test_windows_that_begin_far_outside():
    rng = np.random.default_rng(0)
    lens = [100, 100, 100, 100, 100, 100, 100]
    want = cache_of(rng, lens, 1, 16, 64, "int8")
    cache = pools(want, rng)
    starts = [2 ** 31 - 1, 2 ** 31 - 40, 2 ** 30, 2 ** 30 - 3, -2 ** 31, -1000, 37]
    got = read_all(cache, 200, begin=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    for name in "kv":
        assert not got[name][:6].any()
        assert np.array_equal(got[name][6, :63, 0], want.values(name, 6, 0)[37:])
        assert not got[name][6, 63:].any()
