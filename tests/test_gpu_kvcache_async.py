"""The calls of kvcache.DecodeCache return while the GPU is still busy with what came before
(needs a GPU)."""
from __future__ import annotations

import time

import pytest
import torch

from lossless_bit_level_gb300.kvcache import DecodeCache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [None, [3, 1, 2, 2] * 16])
@pytest.mark.parametrize("max_tokens", [160, 65_536])
def test_no_call_waits_for_the_gpu(max_tokens, counts):
    """Small tables and ones of a megabyte."""
    batch, n = 64, 128
    cache = DecodeCache(n_pages=1000, batch=batch, n_heads=2, head_dim=64, max_tokens=max_tokens,
                        page_tokens=16)
    rows = torch.randn((n, 2, 64), device="cuda").bfloat16()
    q = torch.randn((n, 4, 64), device="cuda").bfloat16()

    def calls():
        for _ in range(9):  # more than a page of each
            cache.append(rows, rows, counts=counts)
            cache.attend(q, 0.125, counts=counts)
        cache.evict(12, 4)

    calls()  # what is allocated or loaded once
    torch.cuda.synchronize()
    lens = list(cache.lengths)
    done = torch.cuda.Event()
    torch.cuda._sleep(1_000_000_000)  # about half a second
    t = time.perf_counter()
    calls()
    host = time.perf_counter() - t
    done.record()
    assert not done.query() and host < 0.25
    torch.cuda.synchronize()
    cache.check()
    each = counts or [2] * batch
    assert cache.lengths == cache.cache.lens.tolist() == [min(n + 9 * c, 12) for n, c in zip(lens, each)]


def test_empty_and_equal_counts_without_offsets():
    """Sequences that hold nothing are evicted and attended; equal counts need no offsets and
    give the same as counts that say so."""
    got = []
    for counts in (None, [5, 5, 5]):
        torch.manual_seed(0)
        cache = DecodeCache(n_pages=12, batch=3, n_heads=2, head_dim=64, max_tokens=64, page_tokens=16)
        cache.evict(8, 2)
        assert cache.lengths == [0, 0, 0] and cache.pages_free == 12
        q = torch.randn((15, 4, 64), device="cuda").bfloat16()
        assert not cache.attend(q[:3], 0.125).any()
        k, v = (torch.randn((15, 2, 64), device="cuda").bfloat16() for _ in range(2))
        cache.append(k, v, counts=counts)
        out = cache.attend(q, 0.125, counts=counts)
        cache.evict(4, 1)
        got.append((out, *cache.read(), cache.weights))
        cache.check()
    for a, b in zip(*got):
        assert torch.equal(a, b)
