"""Bookkeeping of kvcache.DecodeCache on the host (no GPU needed): the pages, tables and
lengths that it hands out, with the cache's tensors in host memory and the library's calls
replaced by ones that only move lengths. Refusals come from the library itself."""
import gc
import weakref

import pytest
import torch

import lossless_bit_level_gb300 as ibp
from lossless_bit_level_gb300 import build_lib, kvcache


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_lib.build()
    return ibp.load()


@pytest.fixture(autouse=True)
def no_stream(monkeypatch):
    monkeypatch.setattr(ibp, "_raw_stream", lambda stream: 0)


def fake_append(cache, k, v, cu=None, new_lens=None, status=None, stream=None):
    n = k.shape[0] // cache.batch
    counts = torch.full((cache.batch,), n, dtype=torch.int32) if cu is None else cu[1:] - cu[:-1]
    new_lens.copy_(cache.lens + counts)


def fake_evict(cache, weights, budget, recent, dst, scratch, new_weights=None, kept=None,
               status=None, stream=None):
    dst.lens.copy_(cache.lens.clamp(max=budget))
    if new_weights is not None:
        new_weights.zero_()


def held(monkeypatch, counts=(40, 40), n_pages=20, max_tokens=160):
    cache = kvcache.DecodeCache(n_pages=n_pages, batch=len(counts), n_heads=1, head_dim=64,
                                max_tokens=max_tokens, page_tokens=16, device="cpu")
    rows = torch.zeros((sum(counts), 1, 64))
    with monkeypatch.context() as m:
        m.setattr(kvcache, "kv_append", fake_append)
        cache.append(rows, rows, counts=counts)
    assert cache.lengths == list(counts) == cache.cache.lens.tolist()
    return cache


def state(cache):
    return cache.pages_free, list(cache.lengths), [list(p) for p in cache._pages], sorted(cache._free), \
        cache.cache.lens.tolist()


def consistent(cache):
    """Every page is free or held by one sequence; the table names those that are held."""
    used = [p for pages in cache._pages for p in pages]
    assert sorted(used + cache._free) == list(range(cache.cache.k_codes.shape[0]))
    P = cache.page_tokens
    for b, pages in enumerate(cache._pages):
        assert len(pages) == -(-cache.lengths[b] // P)
        assert cache.cache.table[b, :len(pages)].tolist() == pages


def test_refused_eviction_keeps_no_pages(monkeypatch):
    cache = held(monkeypatch)
    before = state(cache)
    for budget, recent in ((32, 64), (32, -1), (0, 0), (-5, 0)) * 3:
        with pytest.raises(ibp.IBPError):
            cache.evict(budget, recent)
        assert state(cache) == before
        consistent(cache)
    monkeypatch.setattr(kvcache, "kv_evict", fake_evict)
    cache.evict(32, 16)
    assert cache.lengths == [32, 32] and cache.pages_free == 16
    consistent(cache)


def test_eviction_without_memory_keeps_no_pages(monkeypatch):
    cache = held(monkeypatch)
    before = state(cache)

    def none_left(*a, **kw):
        raise torch.OutOfMemoryError("no memory")

    with monkeypatch.context() as m:
        m.setattr(kvcache, "kv_evict_scratch_bytes", none_left)
        with pytest.raises(torch.OutOfMemoryError):
            cache.evict(32, 16)
    assert state(cache) == before


def test_refused_append_keeps_no_pages(monkeypatch):
    cache = held(monkeypatch, counts=(40, 3))
    before = state(cache)
    good = torch.zeros((80, 1, 64))
    for k, v in ((good, good.half()),                      # types differ
                 (torch.zeros((80, 2, 64)),) * 2,          # heads
                 (torch.zeros((80, 1, 128))[:, :, ::2],) * 2,   # elements apart
                 (good.int(), good.int()),                 # no such type
                 (good, good)):                            # not in device memory
        with pytest.raises((ValueError, ibp.IBPError)):
            cache.append(k, v)
        assert state(cache) == before
        consistent(cache)
    monkeypatch.setattr(kvcache, "kv_append", fake_append)
    cache.append(good[:26], good[:26], counts=[13, 13])
    assert cache.lengths == [53, 16]
    consistent(cache)


def test_what_one_sequence_has_too_many_is_not_anothers(monkeypatch):
    """After a refusal the next call is still checked against the pages that are free."""
    cache = held(monkeypatch, counts=(16, 16), n_pages=6)
    bad = torch.zeros((64, 2, 64))
    with pytest.raises(ValueError):
        cache.append(bad, bad, counts=[64, 0])
    monkeypatch.setattr(kvcache, "kv_append", fake_append)
    rows = torch.zeros((80, 1, 64))
    before = state(cache)
    with pytest.raises(RuntimeError, match="5 pages are needed and 4 are free"):
        cache.append(rows, rows, counts=[0, 80])
    assert state(cache) == before
    cache.append(rows[:64], rows[:64], counts=[0, 64])
    assert cache.lengths == [16, 80] and cache.pages_free == 0
    consistent(cache)


def test_scratch_is_not_kept(monkeypatch):
    """A cache (one for each layer) holds no workspace between calls."""
    cache, seen = held(monkeypatch), []

    def attention(cache, q, out, scale, scratch, **kw):
        seen.append((weakref.ref(scratch), scratch.numel()))

    def evict(cache, weights, budget, recent, dst, scratch, **kw):
        seen.append((weakref.ref(scratch), scratch.numel()))
        fake_evict(cache, weights, budget, recent, dst, scratch, **kw)

    monkeypatch.setattr(kvcache, "kv_attention", attention)
    monkeypatch.setattr(kvcache, "kv_evict", evict)
    cache.attend(torch.zeros((80, 4, 64), dtype=torch.bfloat16), 0.1)
    cache.evict(32, 16)
    gc.collect()
    assert len(seen) == 2 and all(n >= 16 for _, n in seen)
    assert all(ref() is None for ref, _ in seen)
