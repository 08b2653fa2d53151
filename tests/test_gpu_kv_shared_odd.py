"""Attention behind shared beginnings: query rows that are not finite (needs a GPU), for the kernel for
few rows, both halves of the one for many, and all of it. The tolerances are those of
test_gpu_kv_shared.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv_harness import rounded
from test_gpu_kv import check_attention, run_attention
from test_gpu_kv_shared import run_shared, shared_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("answers,each", [(5, 1), (20, 1), (50, 2)])  # 10, 40 and 200 rows a K/V head
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("behind", [True, False])  # tokens of its own behind the beginning, or none
def test_rows_that_are_not_finite_stay_by_themselves(answers, each, dtype, value, behind):
    """One element of one row and head is not finite: with a NaN that row's output is NaN and its sum
    that of a row without tokens, as undivided, and every other row's is right."""
    rng = np.random.default_rng(answers)
    dim = 64
    own = [int(t) for t in rng.integers(0, 60, answers)]
    b = answers // 2
    own[b] = 37 if behind else 0
    groups, counts = [(400, own)], [each] * answers
    want, cache = shared_cache(rng, groups, 1, 16, dim, "int8")
    x = rng.standard_normal((each * answers, 2, dim)).astype(np.float32)
    row = each * b
    x[row, 1, 7] = value
    q = rounded(x, dtype).cuda()
    out, lse = run_shared(cache, groups, q, counts, 0.125)
    if np.isnan(value):
        plain, plain_lse, _, _ = run_attention(cache, q, counts, 0.125, weights=False)
        assert torch.isnan(out[row, 1]).all() and torch.isnan(plain[row, 1]).all()
        assert lse[row, 1] == plain_lse[row, 1] == -np.inf
    x[row, 1] = 0
    q = rounded(x, dtype).cuda()
    clean, clean_lse = run_shared(cache, groups, q, counts, 0.125)
    out[row, 1], lse[row, 1] = clean[row, 1], clean_lse[row, 1]
    check_attention(want, q, counts, 0.125, out, lse, None, None)
