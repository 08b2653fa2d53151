"""Argument checks of attention behind shared beginnings, which answer before any CUDA work (no
GPU needed)."""
import ctypes

import pytest
import torch

import lossless_bit_level_gb300 as ibp
from test_kv_cpu import GEOMETRY, lib, query, struct  # noqa: F401

BIG = 1 << 40


def call(lib, c=None, q=None, groups=1, rows=2, scratch=BIG):  # noqa: F811
    by = ctypes.byref
    return lib.ibp_kv_attention_shared(by(c or struct()), by(q or query()), 16, 16, groups, rows, 16, scratch,
                                       None, None)


@pytest.mark.parametrize("change,code", GEOMETRY)
def test_geometry(lib, change, code):  # noqa: F811
    size = ctypes.c_size_t(0)
    assert call(lib, c=struct(**change)) == code
    assert lib.ibp_kv_attention_shared_scratch_bytes(ctypes.byref(struct(**change)), 2, 1, 4, 1, 2,
                                                     ctypes.byref(size)) == code


@pytest.mark.parametrize("change,code", [
    (dict(dtype=ibp.FP32), ibp.ERR_DTYPE), (dict(q_heads=3), ibp.ERR_ARG), (dict(max_q=2), ibp.ERR_ARG),
    (dict(q_row_stride=20), ibp.ERR_ARG), (dict(out_row_stride=128), ibp.ERR_ARG),
    (dict(scale=float("nan")), ibp.ERR_ARG), (dict(d_weights=16, weights_stride=256), ibp.ERR_ARG),
    (dict(d_weights_in=16), ibp.ERR_ARG), (dict(n_rows=0, max_q=0), ibp.OK),
])
def test_query_refusals(lib, change, code):  # noqa: F811
    assert call(lib, q=query(**change)) == code


@pytest.mark.parametrize("groups,rows", [(-1, 2), (3, 2), (1, -1), (1, (1 << 30) + 1)])
def test_group_refusals(lib, groups, rows):  # noqa: F811
    size = ctypes.c_size_t(0)
    assert call(lib, groups=groups, rows=rows) == ibp.ERR_ARG
    assert lib.ibp_kv_attention_shared_scratch_bytes(ctypes.byref(struct()), 2, 1, 4, groups, rows,
                                                     ctypes.byref(size)) == ibp.ERR_ARG


def test_scratch_and_nulls(lib):  # noqa: F811
    by, size, c = ctypes.byref, ctypes.c_size_t(0), struct()
    for rows, max_q in ((2, 1), (60, 30), (200, 100)):
        n = query(n_rows=rows, max_q=max_q)
        assert lib.ibp_kv_attention_shared_scratch_bytes(by(c), rows, max_q, 4, 1, rows, by(size)) == 0
        assert size.value % 16 == 0 and call(lib, q=n, rows=rows, scratch=size.value - 1) == ibp.ERR_ARG
    assert lib.ibp_kv_attention_shared_scratch_bytes(by(c), 2, 1, 4, 1, 2, None) == ibp.ERR_ARG
    assert lib.ibp_kv_attention_shared(by(c), None, 16, 16, 1, 2, 16, BIG, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_attention_shared(None, by(query()), 16, 16, 1, 2, 16, BIG, None, None) == ibp.ERR_ARG


def test_binding_refusals():
    codes, s = torch.zeros((3, 2, 16, 64), dtype=torch.int8), torch.zeros((3, 2))
    cache = ibp.KVCache(codes, codes, s, s, torch.zeros((2, 4), dtype=torch.int32),
                        torch.zeros(2, dtype=torch.int32))
    q, scratch = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.uint8)
    two, one = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for groups, prefix in ((one, one), (two.long(), one), (two, one.float())):
        with pytest.raises(ValueError):
            ibp.kv_attention_shared(cache, q, torch.zeros_like(q), 1.0, scratch, groups, prefix, 2)
