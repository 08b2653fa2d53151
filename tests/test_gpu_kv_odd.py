"""Attention over the 8-bit cache: query rows that are not finite, and long sequences, for the
kernel for few rows and the one for many (needs a GPU). The tolerances are those of
test_gpu_kv.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv_harness import cache_of, pools, rounded
from test_gpu_kv import check_attention, run_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 12, 130])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_rows_that_are_not_finite_stay_by_themselves(n, dtype, value):
    """One element of one row and head is not finite: with a NaN that row's output is NaN, and
    every other row's is right."""
    rng = np.random.default_rng(n)
    dim, lens, counts = 64, [200, 70], [n, n]
    want = cache_of(rng, lens, 1, 16, dim, "int8")
    cache = pools(want, rng)
    x = rng.standard_normal((2 * n, 2, dim)).astype(np.float32)
    x[n // 2, 1, 7] = value
    out, lse, _, _ = run_attention(cache, rounded(x, dtype).cuda(), counts, 0.125, weights=False)
    if np.isnan(value):
        assert torch.isnan(out[n // 2, 1]).all()
    # the row in question put back: the others are compared as always
    x[n // 2, 1] = 0
    q = rounded(x, dtype).cuda()
    clean, clean_lse, _, _ = run_attention(cache, q, counts, 0.125, weights=False)
    out[n // 2, 1], lse[n // 2, 1] = clean[n // 2, 1], clean_lse[n // 2, 1]
    check_attention(want, q, counts, 0.125, out, lse, None, None)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("n,weights", [(1, True), (3, False), (40, False)])
def test_long_sequences(n, weights, code):
    rng = np.random.default_rng(n)
    lens, counts = [70_001, 20_480, 64], [n, 1, n]
    want = cache_of(rng, lens, 1, 128, 64, code)
    cache = pools(want, rng)
    q = rounded(1.5 * rng.standard_normal((sum(counts), 1, 64)), "bf16").cuda()
    out, lse, w, w_in = run_attention(cache, q, counts, 0.125, weights)
    check_attention(want, q, counts, 0.125, out, lse, w, w_in)
