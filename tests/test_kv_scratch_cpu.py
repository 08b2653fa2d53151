"""Workspace sizes of the 8-bit key/value cache's calls (no GPU needed)."""
import ctypes

import pytest

import lossless_bit_level_gb300 as ibp
from lossless_bit_level_gb300 import build_lib
from test_kv_cpu import struct


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return ibp.load()


def attention_bytes(lib, cache, n_rows, max_q, q_heads, weights):
    size = ctypes.c_size_t(0)
    assert lib.ibp_kv_attention_scratch_bytes(ctypes.byref(cache), n_rows, max_q, q_heads, weights,
                                              ctypes.byref(size)) == 0
    return size.value


@pytest.mark.parametrize("batch,rows,tokens,q_heads,heads", [
    (8, 4096, 4096, 32, 32),          # the prompts of one decoder layer in this repository's size
    (1, 2048, 131_072, 32, 8),        # a chunk of a prompt, with room to grow
    (2, 2048, 120_064, 32, 8),
    (256, 16, 131_072, 32, 8),        # many sequences with room to grow
    (600, 1, 1 << 20, 8, 8),
])
def test_scores_are_held_for_a_bounded_number_of_rows(lib, batch, rows, tokens, q_heads, heads):
    cols = tokens // 64
    cache = struct(batch=batch, n_heads=heads, table_cols=cols, table_stride=cols, n_pages=1 << 20)
    assert attention_bytes(lib, cache, batch * rows, rows, q_heads, 1) <= (1 << 30) + (64 << 20)


def test_what_fits_is_held_for_all_rows(lib):
    """128 rows of 128 heads over 4,096 tokens: as much as the scores of one call take."""
    cache = struct(batch=1, n_heads=128, table_cols=64, table_stride=64)
    n = attention_bytes(lib, cache, 128, 128, 128, 1)
    assert n >= 128 * 128 * 4096 * 4
    assert attention_bytes(lib, cache, 128, 128, 128, 0) < 64 << 20


def test_evictions_scratch_goes_by_what_can_be_kept(lib):
    size = ctypes.c_size_t(0)
    cache = struct(batch=8, n_heads=32, table_cols=64, table_stride=64)
    for budget, kept in ((1, 1), (4095, 4095), (4096, 4096), (10 ** 6, 4096), (1 << 30, 4096)):
        assert lib.ibp_kv_evict_scratch_bytes(ctypes.byref(cache), budget, ctypes.byref(size)) == 0
        assert size.value == 8 * 32 * kept * 8
