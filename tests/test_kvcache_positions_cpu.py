"""Which positions kvcache.DecodeCache rotates new rows by (no GPU needed), with the library's
calls replaced as in test_kvcache_cpu.py: a token's number among all that its sequence was given,
also after evictions, which leave fewer tokens in the cache than that."""
import pytest
import torch

import lossless_bit_level_gb300 as ibp
from lossless_bit_level_gb300 import kvcache
from test_kvcache_cpu import fake_append, fake_evict, lib, no_stream  # noqa: F401


@pytest.fixture
def seen(monkeypatch):
    """Positions that each append with a rotation was given (None: the places in the cache)."""
    got = []

    def fake_rotated(cache, k, v, rotation, positions=None, q=None, q_out=None, cu=None, new_lens=None, status=None):
        got.append(None if positions is None else positions.clone())
        fake_append(cache, k, v, cu=cu, new_lens=new_lens)

    monkeypatch.setattr(kvcache, "kv_append", fake_append)
    monkeypatch.setattr(kvcache, "kv_append_rotated", fake_rotated)
    monkeypatch.setattr(kvcache, "kv_evict", fake_evict)
    return got


def cache_of(batch, **kw):
    return kvcache.DecodeCache(n_pages=60, batch=batch, n_heads=1, head_dim=64, max_tokens=320, page_tokens=16,
                               device="cpu", **kw)


def rotation(axes=1):
    return ibp.KVRotation(torch.zeros((1000, 32, 2)), axis=[i % axes for i in range(32)])


def rows(counts):
    x = torch.zeros((sum(counts), 1, 64))
    return x, x, counts


def test_numbers_go_on_after_an_eviction(seen):
    cache = cache_of(3)
    cache.append(*rows([100, 20, 0]), rotation=rotation())
    assert seen.pop() is None  # places and numbers are the same
    cache.evict(40, 8)
    assert cache.lengths == [40, 20, 0]
    cache.append(*rows([2, 3, 1]), rotation=rotation())
    assert seen.pop().tolist() == [[100], [101], [20], [21], [22], [0]]
    x = torch.zeros((3, 1, 64))
    cache.append(x, x, rotation=rotation(axes=3))  # one each, on every axis
    got = seen.pop()
    assert got.dtype == torch.int32 and got.tolist() == [[102] * 3, [23] * 3, [1] * 3]
    cache.append(*rows([5, 0, 0]))  # rows without a rotation count too
    cache.evict(16, 4)
    cache.append(*rows([1, 1, 1]), rotation=rotation())
    assert seen.pop().tolist() == [[108], [24], [2]]
    own = torch.tensor([[7], [8], [9]], dtype=torch.int32)
    cache.append(*rows([1, 1, 1]), rotation=rotation(), positions=own)
    assert torch.equal(seen.pop(), own)  # given ones are taken
    cache.append(*rows([0, 0, 0]), rotation=rotation())
    assert seen.pop().shape == (0, 1)


def test_an_eviction_that_drops_nothing(seen):
    cache = cache_of(2)
    cache.append(*rows([30, 5]), rotation=rotation())
    cache.evict(64, 8)
    cache.append(*rows([1, 1]), rotation=rotation())
    assert seen == [None, None]


def test_a_refused_append_counts_nothing(seen):
    cache = cache_of(2)
    cache.append(*rows([100, 20]))
    cache.evict(32, 8)
    with pytest.raises(ValueError):
        cache.append(*rows([400, 0]), rotation=rotation())
    cache.append(*rows([1, 1]), rotation=rotation())
    assert seen.pop().tolist() == [[100], [20]]


@pytest.mark.parametrize("evicted", [False, True])
def test_sequences_that_share_go_on_behind_what_they_share(seen, evicted):
    cache = cache_of(3)
    cache.append(*rows([100, 0, 0]))
    if evicted:
        cache.evict(40, 8)  # the kept tokens' last has number 99, in place 39
    tokens = cache.share(0, [1, 2])
    assert tokens == (32 if evicted else 96)
    cache.append(*rows([1, 2, 1]), rotation=rotation())
    # of 40 kept tokens 8 are not shared: number 91 is the highest that a shared one can have
    assert (seen.pop().tolist() == [[100], [92], [93], [92]]) if evicted else seen.pop() is None
