"""Selection of pages where numbers are odd (needs a GPU): query rows with whole runs of NaN.
Columns are compared exactly, as in test_gpu_kv_select.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lossless_bit_level_gb300 as ibp
from kv_harness import cache_of, pools, rounded
from test_gpu_kv import status_word
from test_gpu_kv_select import bounds_of, check_columns, select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [None, 1100])  # one kernel, and two
@pytest.mark.parametrize("rows,group,dim", [(1, 4, 128), (2, 4, 64), (3, 5, 64), (9, 12, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rows_with_runs_of_nan(dtype, rows, group, dim, cols):
    """A NaN counts as 0 wherever it stands, also where it has neighbours: the row's other elements
    set its exponent, and with it what the rows beside it are compared to."""
    rng = np.random.default_rng(rows + group + dim)
    heads = 2
    want = cache_of(rng, [700, 333], heads, 16, dim, "int8")
    cache, status = pools(want, rng, cols=cols), status_word()
    bounds = bounds_of(cache)
    ibp.kv_bounds(cache, bounds, status=status)
    x = rng.standard_normal((2 * rows, heads * group, dim)).astype(np.float32)
    for start, run in ((0, 4), (8, 4), (dim - 4, 4), (1, 11), (0, dim - 5), (0, dim)):
        y = x.copy()
        odd = [rows // 2, rows]  # a row of each sequence
        y[odd, 1::group] *= 20  # larger than those beside it: it chooses the pages
        y[odd, 1::group, start:start + run] = np.nan
        if run == 11:
            y[odd, 1::group, start:start + run:3] = -np.nan
        q = rounded(y, dtype)
        columns = select(cache, bounds, q.cuda(), [rows, rows], 7, status=status)
        check_columns(want, q, [rows, rows], columns)
    assert int(status.item()) == 0
