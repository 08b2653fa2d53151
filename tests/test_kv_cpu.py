"""Argument checks of the 8-bit key/value cache calls, which answer before any CUDA work,
and the plain reference's own rules (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import kv_reference as ref
import lossless_bit_level_gb300 as ibp
from lossless_bit_level_gb300 import build_lib


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return ibp.load()


def struct(**kw):
    base = dict(k_codes=16, v_codes=16, k_scales=16, v_scales=16, d_table=16, d_lens=16,
                n_pages=10, table_stride=4, batch=2, table_cols=4, n_heads=2, page_tokens=64,
                head_dim=128, code=ibp.KV_INT8)
    base.update(kw)
    return ibp.KVCacheStruct(**base)


def rows(**kw):
    base = dict(k=16, v=16, d_cu=None, n_rows=2, k_row_stride=256, k_head_stride=128,
                v_row_stride=256, v_head_stride=128, dtype=ibp.BF16)
    base.update(kw)
    return ibp.KVRows(**base)


def query(**kw):
    base = dict(q=16, out=16, n_rows=2, max_q=1, q_row_stride=512, q_head_stride=128,
                out_row_stride=512, out_head_stride=128, q_heads=4, dtype=ibp.BF16, scale=0.1,
                decay=1.0)
    base.update(kw)
    return ibp.KVQuery(**base)


GEOMETRY = [
    (dict(code=2), ibp.ERR_DTYPE), (dict(head_dim=96), ibp.ERR_UNSUPPORTED),
    (dict(page_tokens=48), ibp.ERR_UNSUPPORTED), (dict(n_heads=0), ibp.ERR_ARG),
    (dict(batch=-1), ibp.ERR_ARG), (dict(table_stride=3), ibp.ERR_ARG),
    (dict(table_cols=1 << 25, table_stride=1 << 25), ibp.ERR_UNSUPPORTED),
    (dict(batch=1 << 17), ibp.ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("change,code", GEOMETRY)
def test_geometry_is_checked_by_every_call(lib, change, code):
    c, ref_, size = struct(**change), ctypes.byref, ctypes.c_size_t(0)
    good = struct()
    assert lib.ibp_kv_append(ref_(c), ref_(rows()), None, None, None) == code
    assert lib.ibp_kv_read(ref_(c), None, 4, 16, 16, ibp.BF16, None, None) == code
    assert lib.ibp_kv_attention_scratch_bytes(ref_(c), 2, 1, 4, 0, ref_(size)) == code
    assert lib.ibp_kv_attention(ref_(c), ref_(query()), 16, 1 << 30, None, None) == code
    assert lib.ibp_kv_evict_scratch_bytes(ref_(c), 5, ref_(size)) == code
    assert lib.ibp_kv_evict(ref_(c), 16, 256, 5, 1, ref_(good), 16, None, 0, None, 16, 1 << 30,
                            None, None) == code
    assert lib.ibp_kv_evict(ref_(good), 16, 256, 5, 1, ref_(c), 16, None, 0, None, 16, 1 << 30,
                            None, None) == code


def test_null_structs(lib):
    size = ctypes.c_size_t(0)
    c = struct()
    assert lib.ibp_kv_append(None, ctypes.byref(rows()), None, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_append(ctypes.byref(c), None, None, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_read(None, None, 4, 16, 16, ibp.BF16, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_attention(ctypes.byref(c), None, 16, 0, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_attention_scratch_bytes(ctypes.byref(c), 2, 1, 4, 0, None) == ibp.ERR_ARG
    assert lib.ibp_kv_evict_scratch_bytes(ctypes.byref(c), 2, None) == ibp.ERR_ARG
    assert lib.ibp_kv_evict(ctypes.byref(c), 16, 256, 5, 1, None, 16, None, 0, None, 16, 1 << 30,
                            None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_attention_scratch_bytes(ctypes.byref(c), 2, 1, 4, 1, ctypes.byref(size)) == 0
    assert size.value > 0 and size.value % 16 == 0


@pytest.mark.parametrize("change,code", [
    (dict(dtype=ibp.W8), ibp.ERR_DTYPE), (dict(n_rows=-1), ibp.ERR_ARG),
    (dict(n_rows=3), ibp.ERR_ARG),            # no offsets: a whole number each
    (dict(k_row_stride=12), ibp.ERR_ARG),     # not whole 16-byte pieces
    (dict(v_head_stride=-128), ibp.ERR_ARG), (dict(k=None), ibp.ERR_ARG),
    (dict(k=24), ibp.ERR_ARG),                # misaligned
    (dict(n_rows=0), ibp.OK),                 # nothing to do
])
def test_append_refusals(lib, change, code):
    assert lib.ibp_kv_append(ctypes.byref(struct()), ctypes.byref(rows(**change)), None, None,
                             None) == code


@pytest.mark.parametrize("change,code", [
    (dict(dtype=ibp.FP32), ibp.ERR_DTYPE), (dict(q_heads=3), ibp.ERR_ARG),
    (dict(q_heads=0), ibp.ERR_ARG), (dict(max_q=-1), ibp.ERR_ARG), (dict(max_q=2), ibp.ERR_ARG),
    (dict(q_row_stride=20), ibp.ERR_ARG), (dict(scale=float("nan")), ibp.ERR_ARG),
    (dict(d_weights_in=16), ibp.ERR_ARG),     # weights in without a place for the result
    (dict(d_weights=16, weights_stride=255), ibp.ERR_ARG),
    (dict(n_rows=0, max_q=0), ibp.OK),
])
def test_attention_refusals(lib, change, code):
    assert lib.ibp_kv_attention(ctypes.byref(struct()), ctypes.byref(query(**change)), 16, 1 << 30,
                                None, None) == code


def test_attention_scratch_too_small(lib):
    c, size = struct(), ctypes.c_size_t(0)
    assert lib.ibp_kv_attention_scratch_bytes(ctypes.byref(c), 2, 1, 4, 0, ctypes.byref(size)) == 0
    assert lib.ibp_kv_attention(ctypes.byref(c), ctypes.byref(query()), 16, size.value - 1, None,
                                None) == ibp.ERR_ARG


def test_read_refusals(lib):
    c = ctypes.byref(struct())
    assert lib.ibp_kv_read(c, None, 4, 16, 16, ibp.W8, None, None) == ibp.ERR_DTYPE
    assert lib.ibp_kv_read(c, None, -1, 16, 16, ibp.BF16, None, None) == ibp.ERR_ARG
    assert lib.ibp_kv_read(c, None, 0, 16, 16, ibp.BF16, None, None) == ibp.OK
    assert lib.ibp_kv_read(c, None, 4, None, None, ibp.BF16, None, None) == ibp.OK


@pytest.mark.parametrize("budget,recent,change,extra", [
    (0, 0, {}, {}), (5, 6, {}, {}), (5, -1, {}, {}),
    (5, 1, dict(n_heads=4), {}), (5, 1, dict(page_tokens=32), {}), (5, 1, dict(batch=3), {}),
    (5, 1, dict(code=ibp.KV_E4M3), {}), (5, 1, dict(head_dim=64), {}),
    (200, 1, dict(table_cols=3), {}),         # the destination cannot hold the budget
    (5, 1, {}, dict(stride=255)), (5, 1, {}, dict(new=16, new_stride=4)),
    (5, 1, {}, dict(scratch=8)),
])
def test_evict_refusals(lib, budget, recent, change, extra):
    assert lib.ibp_kv_evict(ctypes.byref(struct()), 16, extra.get("stride", 256), budget, recent,
                            ctypes.byref(struct(**change)), 16, extra.get("new"),
                            extra.get("new_stride", 0), None, 16, extra.get("scratch", 1 << 30),
                            None, None) == ibp.ERR_ARG


def test_binding_refusals():
    codes = torch.zeros((3, 2, 16, 64), dtype=torch.int8)
    s, table = torch.zeros((3, 2)), torch.zeros((2, 4), dtype=torch.int32)
    lens = torch.zeros(2, dtype=torch.int32)
    good = ibp.KVCache(codes, codes.clone(), s, s.clone(), table, lens)
    assert (good.batch, good.capacity, good.n_heads) == (2, 64, 2)
    for bad in ((codes.float(), codes, s, s, table, lens), (codes, codes[:2], s, s, table, lens),
                (codes, codes, s[:2], s, table, lens), (codes, codes, s, s, table.long(), lens),
                (codes, codes, s, s, table, lens[:1]),
                (codes.transpose(1, 2).contiguous().transpose(1, 2),) * 2 + (s, s, table, lens)):
        with pytest.raises(ValueError):
            ibp.KVCache(*bad)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    x = torch.zeros((2, 2, 64))
    for call in (lambda: ibp.kv_append(good, x[:, :1], x),
                 lambda: ibp.kv_append(good, x, x.half()),
                 lambda: ibp.kv_append(good, x, x, cu=torch.zeros(2, dtype=torch.int32)),
                 lambda: ibp.kv_read(good, x, None),
                 lambda: ibp.kv_attention(good, q, q.half(), 1.0, x),
                 lambda: ibp.kv_attention(good, q, q, 1.0, x,
                                          cu_q=torch.zeros(3, dtype=torch.int32)),
                 lambda: ibp.kv_attention(good, q, q, 1.0, x, weights=torch.zeros((2, 1, 64))),
                 lambda: ibp.kv_evict(good, torch.zeros((2, 64)), 4, 1, good, x)):
        with pytest.raises(ValueError):
            call()


def test_reference_e4m3_matches_the_stored_type():
    """The reference's e4m3 rounding and its value table against torch's own type."""
    y = np.concatenate([np.linspace(-448, 448, 20011), np.ldexp(1.0, np.arange(-14, 9)),
                        np.ldexp(1.5, np.arange(-14, 8)) * 1.0625]).astype(np.float32)
    t = torch.from_numpy(y).to(torch.float8_e4m3fn)
    assert np.array_equal(ref.e4m3_round(y), t.float().numpy().astype(np.float64))
    values = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(ref.e4m3_values(), values.float().numpy(), equal_nan=True)


def test_reference_append_in_pieces():
    """Rows in one piece or token by token: the same lengths, and values within the
    rounding of the larger scale (each rescaling rounds once more)."""
    rng = np.random.default_rng(0)
    x = {n: rng.standard_normal((40, 2, 64)).astype(np.float32) for n in "kv"}
    a, b = ref.Cache(1, 2, 16, 64, "int8"), ref.Cache(1, 2, 16, 64, "int8")
    a.append(0, x)
    for i in range(40):
        b.append(0, {n: v[i:i + 1] for n, v in x.items()})
    assert a.lens == b.lens == [40]
    for h in range(2):
        scale = max(s for s, _ in a.tiles["k"][0][h])
        assert np.abs(a.values("k", 0, h) - x["k"][:, h]).max() <= scale * 0.51
        # at most 15 later scales, each of which may round by half a step again
        assert np.abs(b.values("k", 0, h) - x["k"][:, h]).max() <= scale * 0.51 * 16
