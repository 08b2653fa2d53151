"""Eviction of codes and scales that no append writes, in a pool that a caller fills (needs a
GPU): NaN codes of e4m3, page scales that are NaN or infinite. The rule stays the header's: a
page's scale comes from its largest finite magnitude, NaN becomes code 0, an infinity the
largest code of its sign. Compared exactly."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref
import lossless_bit_level_gb300 as ibp
from kv_harness import cache_of, pools, read_all
from test_gpu_kv import status_word

pytestmark = pytest.mark.gpu


def spoil(cache, rng, codes, scales):
    """A NaN code in about every fifth token; some pages' scales NaN or infinite."""
    for name in "kv":
        for b in range(cache.batch):
            for h in range(cache.heads):
                tiles = cache.tiles[name][b][h]
                for j, (s, c) in enumerate(tiles):
                    if codes:
                        hit = rng.random(c.shape[0]) < 0.2
                        c[hit, rng.integers(0, c.shape[1], hit.sum())] = np.nan
                    if scales:
                        s = np.float32(rng.choice([s, s, s, np.nan, np.inf]))
                    tiles[j] = (s, c)


@pytest.mark.filterwarnings("ignore:invalid value")
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (64, 128)])
@pytest.mark.parametrize("code,codes,scales", [("e4m3", True, False), ("e4m3", True, True),
                                               ("int8", False, True)])
def test_evict_values_that_are_not_finite(code, codes, scales, dim, page):
    rng = np.random.default_rng(dim + page)
    lens, heads, budget, recent = [300, 45, 150], 2, 100, 17
    src = cache_of(rng, lens, heads, page, dim, code)
    spoil(src, rng, codes, scales)
    cache = pools(src, rng)
    w = [[rng.random(n).astype(np.float32) for _ in range(heads)] for n in lens]
    wt = np.zeros((len(lens), heads, cache.capacity), np.float32)
    for b, n in enumerate(lens):
        for h in range(heads):
            wt[b, h, :n] = w[b][h]
    want, _ = src.evict(w, budget, recent)
    dst = pools(ref.Cache(len(lens), heads, page, dim, code), rng, room=budget)
    scratch = torch.empty(ibp.kv_evict_scratch_bytes(cache, budget), dtype=torch.uint8, device="cuda")
    status = status_word()
    ibp.kv_evict(cache, torch.from_numpy(wt).cuda(), budget, recent, dst, scratch, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = read_all(dst, budget)
    for b, n in enumerate(want.lens):
        for h in range(heads):
            for name in "kv":
                assert np.array_equal(got[name][b, :n, h], want.values(name, b, h)), (name, b, h)
