"""Argument checks of the append with a rotation, which answer before any CUDA work, and the
plain rotation's own rules (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import kv_rotate_reference as turn
import lossless_bit_level_gb300 as ibp
from test_kv_cpu import GEOMETRY, lib, rows, struct  # noqa: F401


def rotation(**kw):
    base = dict(d_table=16, d_positions=None, n_positions=100, dim=128, axes=1, interleaved=0)
    axis = kw.pop("axis", [0] * 64)
    base.update(kw)
    return ibp.KVRotationStruct(*base.values(), (ctypes.c_uint8 * 64)(*axis))


def turned(**kw):
    base = dict(q=16, out=1 << 20, q_row_stride=512, q_head_stride=128, out_row_stride=512,
                out_head_stride=128, q_heads=4)
    base.update(kw)
    return ibp.KVTurned(**base)


def call(lib, c=None, r=None, t=None, q=None):  # noqa: F811
    by = ctypes.byref
    return lib.ibp_kv_append_rotated(by(c or struct()), by(r or rows()), by(t or rotation()),
                                     by(q) if q else None, None, None, None)


@pytest.mark.parametrize("change,code", GEOMETRY)
def test_geometry(lib, change, code):  # noqa: F811
    assert call(lib, c=struct(**change)) == code


@pytest.mark.parametrize("change", [
    dict(dim=8), dict(dim=0), dict(dim=24), dict(dim=144), dict(dim=-16), dict(axes=0), dict(axes=5),
    dict(axis=[0] * 63 + [1]), dict(axes=2, axis=[2] * 64), dict(n_positions=0), dict(n_positions=-1),
    dict(n_positions=(1 << 30) + 1),
])
def test_rotation_refusals(lib, change):  # noqa: F811
    assert call(lib, t=rotation(**change)) == ibp.ERR_ARG
    # the pairs past dim are not looked at, and nothing to do is no error
    assert call(lib, r=rows(n_rows=0), t=rotation(dim=64, axis=[0] * 32 + [9] * 32)) == ibp.OK
    assert call(lib, r=rows(n_rows=0), t=rotation(**change)) == ibp.ERR_ARG


@pytest.mark.parametrize("change", [
    dict(q_heads=0), dict(q_heads=70_000), dict(q_row_stride=20), dict(out_head_stride=-8),
    dict(out_row_stride=128), dict(out_head_stride=64), dict(out_head_stride=0),
])
def test_query_refusals(lib, change):  # noqa: F811
    assert call(lib, q=turned(**change)) == ibp.ERR_ARG


def test_rows_and_null_refusals(lib):  # noqa: F811
    by = ctypes.byref
    assert call(lib, r=rows(dtype=ibp.W8)) == ibp.ERR_DTYPE
    assert call(lib, r=rows(n_rows=3)) == ibp.ERR_ARG
    assert call(lib, r=rows(k=24)) == ibp.ERR_ARG
    assert lib.ibp_kv_append_rotated(by(struct()), by(rows()), None, None, None, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_append_rotated(by(struct()), None, by(rotation()), None, None, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_append_rotated(None, by(rows()), by(rotation()), None, None, None, None) == ibp.ERR_ARG


def test_binding_refusals():
    table = torch.zeros((10, 32, 2))
    for bad in (table[:, :, :1], table.half(), table[::2], table[0]):
        with pytest.raises(ValueError):
            ibp.KVRotation(bad)
    for axis in ([0] * 31, [4] * 32, [-1] * 32):
        with pytest.raises(ValueError):
            ibp.KVRotation(table, axis=axis)
    r = ibp.KVRotation(table, axis=[0] * 16 + [2] * 16)
    assert r.axes == 3
    codes, s = torch.zeros((3, 2, 16, 64), dtype=torch.int8), torch.zeros((3, 2))
    cache = ibp.KVCache(codes, codes, s, s, torch.zeros((2, 4), dtype=torch.int32),
                        torch.zeros(2, dtype=torch.int32))
    k, q = torch.zeros((2, 2, 64)), torch.zeros((2, 4, 64))
    for kw in (dict(positions=torch.zeros((2, 2), dtype=torch.int32)), dict(positions=torch.zeros((2, 3))),
               dict(q=q[:1]), dict(q=q.half()), dict(q=q, q_out=k), dict(q_out=q), dict(v=k[:1])):
        with pytest.raises(ValueError):
            ibp.kv_append_rotated(cache, k, kw.pop("v", k), r, **kw)


def test_rotation_table_on_the_host():
    t = ibp.rotation_table(70_000, 64, base=500.0, device="cpu").numpy()
    angle = 69_999 * 500.0 ** (-np.arange(32) / 32)
    assert np.allclose(t[69_999], np.stack([np.cos(angle), np.sin(angle)], 1), rtol=0, atol=2.0 ** -24 + 1e-10)
    # a rotation keeps each pair's length and adds up over positions: a tolerance of a few
    # roundings of 2^-24 of values near 1
    x = np.random.default_rng(0).standard_normal((1, 1, 64)).astype(np.float32)
    at = lambda p: np.array([[p]])  # noqa: E731
    for inter in (False, True):
        once = turn.rotated(x, t, at(30), [0] * 32, inter)
        twice = turn.rotated(turn.rotated(x, t, at(10), [0] * 32, inter), t, at(20), [0] * 32, inter)
        assert np.allclose(once, twice, rtol=0, atol=16 * 2.0 ** -24 * np.abs(x).max())
