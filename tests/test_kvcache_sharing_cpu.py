"""Bookkeeping of shared beginnings in kvcache.DecodeCache on the host (no GPU needed), with the
library's calls replaced as in test_kvcache_cpu.py."""
import pytest
import torch

import lossless_bit_level_gb300 as ibp
from lossless_bit_level_gb300 import kvcache
from test_kvcache_cpu import fake_append, fake_evict, lib, no_stream  # noqa: F401


def cache_of(monkeypatch, batch=5, n_pages=40, **kw):
    monkeypatch.setattr(kvcache, "kv_append", fake_append)
    return kvcache.DecodeCache(n_pages=n_pages, batch=batch, n_heads=1, head_dim=64, max_tokens=160,
                               page_tokens=16, device="cpu", **kw)


def rows(counts):
    x = torch.zeros((sum(counts), 1, 64))
    return x, x, counts


def test_shared_pages_are_held_once_and_freed_once(monkeypatch):
    cache = cache_of(monkeypatch)
    cache.append(*rows([0, 40, 0, 0, 0]))
    assert cache.share(1, [2, 3]) == 32
    assert cache.lengths == [0, 40, 32, 32, 0] == cache.cache.lens.tolist()
    assert cache.pages_free == 40 - 3
    begin = cache._pages[1][:2]
    assert cache._pages[2] == cache._pages[3] == begin
    cache.append(*rows([5, 1, 20, 0, 7]))
    assert cache.lengths == [5, 41, 52, 32, 7]
    for b, pages in enumerate(cache._pages):
        assert len(pages) == -(-cache.lengths[b] // 16)
        assert cache.cache.table[b, :len(pages)].tolist() == pages
    own = [p for pages in cache._pages for p in pages if p not in begin]
    assert len(own) == len(set(own)) and not set(own) & set(begin)
    offsets, prefix = cache._shared()
    assert offsets.tolist() == [0, 1, 4] and prefix.tolist() == [0, 32]
    monkeypatch.setattr(kvcache, "kv_evict", fake_evict)
    cache.evict(16, 4)
    assert cache.lengths == [5, 16, 16, 16, 7]
    used = [p for pages in cache._pages for p in pages]
    assert sorted(used + cache._free) == list(range(40)) and not cache._groups


def test_refusals(monkeypatch):
    cache = cache_of(monkeypatch)
    cache.append(*rows([40, 0, 0, 0, 3]))
    for src, wanted in ((0, []), (0, [2]), (0, [1, 3]), (3, [4]), (-1, [0]), (4, [5]), (0, [1, 2, 3, 4])):
        with pytest.raises(ValueError):
            cache.share(src, wanted)
    assert cache.share(0, [1]) == 32
    for src, wanted in ((0, [1]), (1, [2])):
        with pytest.raises(ValueError):
            cache.share(src, wanted)
    assert cache.share(2, [3]) == 0 and cache.lengths == [40, 32, 0, 0, 3]  # nothing to share
    with pytest.raises(ValueError):
        cache.append(*rows([1] * 5), q=torch.zeros((5, 1, 64)))
    with pytest.raises(RuntimeError):
        cache.attend(torch.zeros((5, 1, 64), dtype=torch.bfloat16), 1.0, pages=4)


def test_what_an_attending_step_calls(monkeypatch):
    """Shared beginnings go to the shared call where no weights are kept, selected pages to
    selection, everything else to the plain call."""
    seen = []
    for name in ("kv_attention", "kv_attention_shared", "kv_attention_selected", "kv_select", "kv_bounds"):
        monkeypatch.setattr(kvcache, name, lambda *a, name=name, **kw: seen.append((name, kw)))
    q = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    for track in (False, True):
        cache = cache_of(monkeypatch, track_weights=track, track_bounds=True)
        cache.append(*rows([64, 0, 0, 0, 0]))
        assert seen.pop()[0] == "kv_bounds"
        cache.attend(q, 0.1)
        assert [n for n, _ in seen] == ["kv_attention"]
        cache.share(0, [1, 2, 3])
        cache.append(*rows([1] * 5))
        seen.clear()
        cache.attend(q, 0.1)
        assert [n for n, _ in seen] == ["kv_attention" if track else "kv_attention_shared"]
        seen.clear()
        cache.attend(q, 0.1, pages=3)
        assert [n for n, _ in seen] == ["kv_select", "kv_attention_selected"]
        seen.clear()
