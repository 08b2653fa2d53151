"""Workspace sizes of the 8-bit key/value cache's calls (no GPU needed)."""
import ctypes

import pytest

import lossless_bit_level_gb300 as ibp
from lossless_bit_level_gb300 import build_lib
from test_kv_cpu import query, struct


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


def test_rows_a_sequence_are_bounded_by_all_rows(lib):
    """max_q is a bound that a caller may set high: it changes nothing past n_rows, and one
    that cannot be meant is refused."""
    size = ctypes.c_size_t(0)
    cache = struct(batch=4, n_heads=2)
    for weights in (0, 1):
        few = attention_bytes(lib, cache, 6, 6, 4, weights)
        assert attention_bytes(lib, cache, 6, 1 << 20, 4, weights) == few
        for max_q in ((1 << 30) + 1, 1 << 33, 1 << 62, (1 << 63) - 1):
            assert lib.ibp_kv_attention_scratch_bytes(ctypes.byref(cache), 6, max_q, 4, weights,
                                                      ctypes.byref(size)) == ibp.ERR_ARG
    # 2^32 (row, head) pairs of a K/V head: more than the kernels count
    assert lib.ibp_kv_attention_scratch_bytes(ctypes.byref(struct(n_heads=1)), 1 << 20, 1 << 20, 4096,
                                              0, ctypes.byref(size)) == ibp.ERR_UNSUPPORTED


def test_a_bound_that_overflows_is_refused(lib):
    """4 * 2^62 is 0 in 64 bits: no rows of no sequence."""
    q = query(n_rows=0, max_q=1 << 62, d_cu=None, d_weights=16, weights_stride=256)
    assert lib.ibp_kv_attention(ctypes.byref(struct(batch=4)), ctypes.byref(q), 16, 1 << 40, None,
                                None) == ibp.ERR_ARG
