"""Attention of many query rows where every CTA goes over seven or ten tiles of several
segments, so that every barrier and place in tensor memory is used again and again (needs a
GPU). The tolerances are those of test_gpu_kv.py; repeated calls give equal bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv_harness import cache_of, pools, rounded
from test_gpu_kv import check_attention, run_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,counts,q_heads,heads,dim,page,code,dtype", [
    ([8192, 3001], [130, 257], 16, 8, 128, 64, "int8", "bf16"),
    ([9000, 100, 2500], [256, 90, 40], 12, 12, 64, 16, "e4m3", "fp16"),
])
def test_long_stretches(lens, counts, q_heads, heads, dim, page, code, dtype):
    rng = np.random.default_rng(sum(lens))
    want = cache_of(rng, lens, heads, page, dim, code)
    # scores that grow along the sequence: references are raised in every stretch
    for b in range(len(lens)):
        for h in range(heads):
            tiles = want.tiles["k"][b][h]
            for j, (s, c) in enumerate(tiles):
                tiles[j] = (np.float32(s * (0.5 + 2.5 * j / len(tiles))), c)
    cache = pools(want, rng)
    q = rounded(1.5 * rng.standard_normal((sum(counts), q_heads, dim)), dtype).cuda()
    out, lse, _, _ = run_attention(cache, q, counts, 1 / np.sqrt(dim), weights=False)
    check_attention(want, q, counts, 1 / np.sqrt(dim), out, lse, None, None)
    for _ in range(10):
        again = run_attention(cache, q, counts, 1 / np.sqrt(dim), weights=False)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
