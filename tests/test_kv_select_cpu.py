"""Argument checks of page selection and of attention over selected pages, which answer before
any CUDA work, and the plain rules' own (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import kv_reference as ref
import kv_select_reference as sel
import lossless_bit_level_gb300 as ibp
from test_kv_cpu import GEOMETRY, lib, query, struct  # noqa: F401

BIG = 1 << 40


@pytest.mark.parametrize("change,code", GEOMETRY)
def test_geometry(lib, change, code):  # noqa: F811
    c, by, size = struct(**change), ctypes.byref, ctypes.c_size_t(0)
    assert lib.ibp_kv_bounds(by(c), 16, None, None, None) == code
    assert lib.ibp_kv_select_scratch_bytes(by(c), by(size)) == code
    assert lib.ibp_kv_select(by(c), 16, by(query()), 4, 16, 16, BIG, None, None) == code
    assert lib.ibp_kv_attention_selected_scratch_bytes(by(c), 2, 1, 4, 4, by(size)) == code
    assert lib.ibp_kv_attention_selected(by(c), by(query()), 16, 4, 16, BIG, None, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(dtype=ibp.FP32), ibp.ERR_DTYPE), (dict(q_heads=3), ibp.ERR_ARG), (dict(q_heads=0), ibp.ERR_ARG),
    (dict(max_q=-1), ibp.ERR_ARG), (dict(max_q=2), ibp.ERR_ARG), (dict(q_row_stride=20), ibp.ERR_ARG),
    (dict(n_rows=2, max_q=0), ibp.ERR_ARG),
])
def test_query_refusals(lib, change, code):  # noqa: F811
    by, c = ctypes.byref, struct()
    assert lib.ibp_kv_select(by(c), 16, by(query(**change)), 4, 16, 16, BIG, None, None) == code
    assert lib.ibp_kv_attention_selected(by(c), by(query(**change)), 16, 4, 16, BIG, None, None) == code


@pytest.mark.parametrize("change", [
    dict(scale=float("nan")), dict(out_row_stride=20), dict(out_row_stride=128), dict(out_head_stride=64),
    dict(d_weights=16, weights_stride=256), dict(d_weights_in=16),
])
def test_attention_refusals(lib, change):  # noqa: F811
    by = ctypes.byref
    assert lib.ibp_kv_attention_selected(by(struct()), by(query(**change)), 16, 4, 16, BIG, None,
                                         None) == ibp.ERR_ARG


@pytest.mark.parametrize("max_q,least", [(1, 2), (2, 3), (65, 3), (66, 4), (0, 1)])
def test_lists_hold_the_first_page_and_the_rows_own(lib, max_q, least):  # noqa: F811
    by, size, c = ctypes.byref, ctypes.c_size_t(0), struct()
    for pages, code in ((least - 1, ibp.ERR_ARG), (least, ibp.OK), ((1 << 24) + 1, ibp.ERR_ARG)):
        assert lib.ibp_kv_attention_selected_scratch_bytes(by(c), 2 * max_q, max_q, 4, pages, by(size)) == code
    q = query(n_rows=2 * max_q, max_q=max_q)
    assert lib.ibp_kv_select(by(c), 16, by(q), least - 1, 16, 16, BIG, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_attention_selected(by(c), by(q), 16, least - 1, 16, BIG, None, None) == ibp.ERR_ARG


def test_scratch_and_nulls(lib):  # noqa: F811
    by, size, c = ctypes.byref, ctypes.c_size_t(0), struct()
    assert lib.ibp_kv_select_scratch_bytes(by(c), by(size)) == 0
    assert size.value == 2 * 2 * 4 * 4  # a float for every sequence, head and column
    assert lib.ibp_kv_select(by(c), 16, by(query()), 4, 16, 16, size.value - 1, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_attention_selected_scratch_bytes(by(c), 2, 1, 4, 4, by(size)) == 0
    assert lib.ibp_kv_attention_selected(by(c), by(query()), 16, 4, 16, size.value - 1, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_select_scratch_bytes(by(c), None) == ibp.ERR_ARG
    assert lib.ibp_kv_select(by(c), 16, None, 4, 16, 16, BIG, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_attention_selected(by(c), None, 16, 4, 16, BIG, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_bounds(None, 16, None, None, None) == ibp.ERR_ARG
    none = query(n_rows=0, max_q=0)
    assert lib.ibp_kv_attention_selected(by(c), by(none), 16, 4, 16, BIG, None, None) == ibp.OK
    assert lib.ibp_kv_bounds(by(struct(batch=0)), 16, None, None, None) == ibp.OK


def test_binding_refusals():
    codes, s = torch.zeros((3, 2, 16, 64), dtype=torch.int8), torch.zeros((3, 2))
    cache = ibp.KVCache(codes, codes, s, s, torch.zeros((2, 4), dtype=torch.int32),
                        torch.zeros(2, dtype=torch.int32))
    q, scratch = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.uint8)
    for bad in (torch.zeros((3, 2, 2, 64)), torch.zeros((3, 2, 64), dtype=torch.int8),
                torch.zeros((4, 2, 2, 64), dtype=torch.int8)):
        with pytest.raises(ValueError):
            ibp.kv_bounds(cache, bad)
    good = torch.zeros((3, 2, 2, 64), dtype=torch.int8)
    for bad in (torch.zeros((2, 2, 4)), torch.zeros((2, 4), dtype=torch.int32),
                torch.zeros((2, 1, 4), dtype=torch.int32)):
        with pytest.raises(ValueError):
            ibp.kv_select(cache, good, q, bad, scratch)
        with pytest.raises(ValueError):
            ibp.kv_attention_selected(cache, bad, q, torch.zeros_like(q), 1.0, scratch)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_a_pages_score_is_above_each_of_its_tokens(code):
    """The plain rule: no token's product with the rounded query passes its page's score."""
    rng = np.random.default_rng(0)
    cache = ref.Cache(1, 1, 16, 64, code)
    cache.append(0, {n: (3 * rng.standard_normal((100, 1, 64))).astype(np.float32) for n in "kv"})
    row = rng.standard_normal((1, 64)).astype(np.float32)
    n, e = sel.whole(row[0])
    k = cache.values("k", 0, 0).astype(np.float64)
    got = sel.scores(cache, 0, 0, row).astype(np.float64)
    # a page's scale is that of its codes; e4m3's bounds are in units of 448/127 of a code
    unit = 1.0 if code == "int8" else 448.0 / 127.0
    for j in range(7):
        best = (k[16 * j:16 * j + 16] @ n).max() * 2.0 ** (e - 6)
        assert got[j] * unit * (1 + 2.0 ** -22) + 1e-12 >= best
    assert sel.columns(cache, 0, 0, row, 1, 7) == list(range(7))
    some = sel.columns(cache, 0, 0, row, 1, 3)
    assert some[0] == 0 and some[-1] == 6 and len(some) == 3
