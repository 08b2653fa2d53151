"""Eviction from long lists, exactly against the plain reference (needs a GPU): lists shared by
a cluster of 2, 4 and 8 CTAs, lists whose keys do not fit their CTAs' shared memory, with one
CTA and with eight to a list; weights with ties, all equal, and with NaN, infinities, zeros of
both signs and denormals."""
from __future__ import annotations

import pytest

import test_gpu_kv

pytestmark = pytest.mark.gpu

LISTS = [
    # (lengths, heads, page, code, budget, recent)
    ([9_000], 1, 16, "int8", 2_345, 100),                  # a cluster of two
    ([17_000, 8_500], 2, 64, "e4m3", 5_000, 0),            # of four
    ([70_000, 3_000, 41_007], 1, 128, "int8", 12_345, 777),  # of eight
    ([200_001], 1, 128, "int8", 60_001, 60_000),           # of eight, keys read from memory each time
    ([26_001] + [5] * 50 + [1_000] * 29, 1, 128, "int8", 900, 64),  # a lone CTA, the same
]


@pytest.mark.parametrize("lens,heads,page,code,budget,recent", LISTS)
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd"])
def test_long_lists(lens, heads, page, code, budget, recent, kind):
    test_gpu_kv.test_evict_is_exact(lens, heads, page, 64, code, budget, recent, kind)


@pytest.mark.parametrize("budget", [300, 320, 321, 100_000])
def test_budgets_around_and_past_the_capacity(budget):
    test_gpu_kv.test_evict_is_exact([300, 0, 17], 2, 64, 64, "int8", budget, 9, "random")
