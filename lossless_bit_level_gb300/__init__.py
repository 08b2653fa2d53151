"""Python binding of the GB300 Invariant Bit Packing codec (``include/ibp.h``).

Argument marshalling only: every step of the codec runs in the CUDA kernels of
``_build/libibp_gb300.so``. Tensors are torch tensors used as plain memory
(device memory, or page-locked host memory for rows and slots read or written
zero-copy); calls are enqueued on the current CUDA stream unless one is given.
There is no CPU fallback: importing works without the library, but every call
raises if the shared library has not been built (``build_lib.build()``).

Method: "Reducing the GPU Memory Bottleneck with Lossless Compression for ML --
Extended", technical summary, "Core algorithm" and "System integration".

The path, in order:
  build_meta (or meta_count + meta_finalize across holders; build_meta_select for
  the saving-aware mask)       -> 16-byte metadata in device memory
  compress                     -> fixed-size slots + bitmask (+ row sizes)
  decompress_gather            -> the rows an index list names, rebuilt bit for bit
Gather variants: decompress_gather_dedup (each distinct row read once),
decompress_gather_sized (only each row's used bytes), decompress_gather_batched
(several tables in one launch), decompress_range (rows in order). Next to them: the
packed store (pack_offsets, pack, decompress_gather_packed) and per-position or
block-position metadata (build_meta_positions, build_meta_block_positions,
compress_positions, decompress_gather_positions). Beside the codec, an 8-bit paged
key/value cache for the K/V rows it stores: KVCache, kv_append, kv_read, kv_attention,
kv_evict; kv_append_rotated (positions rotated on the way in), kv_attention_shared (beginnings
that sequences share), kv_bounds, kv_select and kv_attention_selected (a few pages of many)
(``kvcache.py`` manages one). ``offload.py`` streams compressed
tensors through device buffers; ``sharded.py`` builds the metadata of a table spread
over several processes.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import build_lib

FP32, FP16, BF16, W8 = 0, 1, 2, 3
KV_INT8, KV_E4M3 = 0, 1
OK = 0
ERR_ARG, ERR_DTYPE, ERR_UNSUPPORTED, ERR_CUDA, ERR_INDEX, ERR_CORRUPT, ERR_META, ERR_TIMEOUT = (
    -1, -2, -3, -4, -5, -6, -7, -8)

_TORCH_DTYPES = {torch.float32: FP32, torch.float16: FP16, torch.bfloat16: BF16}
for _name in ("float8_e4m3fn", "float8_e5m2"):
    if hasattr(torch, _name):
        _TORCH_DTYPES[getattr(torch, _name)] = W8
WIDTH = {FP32: 32, FP16: 16, BF16: 16, W8: 8}

_lib = None


class IBPError(RuntimeError):
    def __init__(self, code: int, call: str):
        self.code = code
        super().__init__(f"{call}: {status_string(code)} ({code})")


class GatherJob(ctypes.Structure):
    """ibp_gather_job: one gather of a batch."""
    _fields_ = [("slots", ctypes.c_void_p), ("slot_bytes", ctypes.c_int64),
                ("n_rows", ctypes.c_int64), ("d_row_bitmask", ctypes.c_void_p),
                ("d_meta", ctypes.c_void_p), ("d_idx", ctypes.c_void_p),
                ("n_idx", ctypes.c_int64), ("out", ctypes.c_void_p)]


class Stats(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int64), ("n_compressed", ctypes.c_int64),
                ("raw_bytes", ctypes.c_int64), ("stored_bytes", ctypes.c_int64),
                ("total_bits", ctypes.c_int64)]


class KVCacheStruct(ctypes.Structure):
    """ibp_kv_cache"""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("d_table", ctypes.c_void_p), ("d_lens", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("table_stride", ctypes.c_int64),
                ("batch", ctypes.c_int32), ("table_cols", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("code", ctypes.c_int32)]


class KVRows(ctypes.Structure):
    """ibp_kv_rows"""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("d_cu", ctypes.c_void_p),
                ("n_rows", ctypes.c_int64), ("k_row_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("v_row_stride", ctypes.c_int64),
                ("v_head_stride", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class KVQuery(ctypes.Structure):
    """ibp_kv_query"""
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("d_lse", ctypes.c_void_p),
                ("d_cu", ctypes.c_void_p), ("d_weights_in", ctypes.c_void_p),
                ("d_weights", ctypes.c_void_p), ("n_rows", ctypes.c_int64),
                ("max_q", ctypes.c_int64), ("weights_stride", ctypes.c_int64),
                ("q_row_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("q_heads", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("decay", ctypes.c_float)]


class KVRotationStruct(ctypes.Structure):
    """ibp_kv_rotation"""
    _fields_ = [("d_table", ctypes.c_void_p), ("d_positions", ctypes.c_void_p),
                ("n_positions", ctypes.c_int64), ("dim", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("axis", ctypes.c_uint8 * 64)]


class KVTurned(ctypes.Structure):
    """ibp_kv_turned"""
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("q_row_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("q_heads", ctypes.c_int32)]


SYMBOLS = ("ibp_status_string", "ibp_slot_bytes", "ibp_meta_scratch_bytes", "ibp_build_meta",
           "ibp_compress", "ibp_decompress_gather", "ibp_query", "ibp_probe_read",
           "ibp_build_meta_noalloc", "ibp_meta_select_scratch_bytes", "ibp_build_meta_select",
           "ibp_pack_scratch_bytes", "ibp_pack_offsets", "ibp_pack", "ibp_decompress_gather_packed",
           "ibp_decompress_range", "ibp_meta_positions_scratch_bytes", "ibp_build_meta_positions",
           "ibp_compress_positions", "ibp_decompress_gather_positions",
           "ibp_decompress_gather_sized", "ibp_decompress_gather_batched", "ibp_meta_count",
           "ibp_meta_finalize", "ibp_build_meta_block_positions", "ibp_gather_dedup_scratch_bytes",
           "ibp_decompress_gather_dedup", "ibp_query_async", "ibp_kv_append", "ibp_kv_read",
           "ibp_kv_attention_scratch_bytes", "ibp_kv_attention", "ibp_kv_evict_scratch_bytes",
           "ibp_kv_evict", "ibp_kv_append_rotated", "ibp_kv_bounds",
           "ibp_kv_select_scratch_bytes", "ibp_kv_select",
           "ibp_kv_attention_selected_scratch_bytes", "ibp_kv_attention_selected",
           "ibp_kv_attention_shared_scratch_bytes", "ibp_kv_attention_shared")

# declared in include/ibp_testing.h (a testing hook, not part of the codec)
TESTING_SYMBOLS = ("ibp_testing_set_wait_limit_ns", "ibp_testing_withhold_plans")

MAX_MASK_CANDIDATES = 33


def library_path() -> str:
    return build_lib.LIB


def load() -> ctypes.CDLL:
    """Load the built library (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    path = build_lib.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"IBP CUDA library not built ({path}); run "
                           "lossless_bit_level_gb300.build_lib.build() first")
    lib = ctypes.CDLL(path)
    i64, i32, u32, dbl, vp = (ctypes.c_int64, ctypes.c_int, ctypes.c_uint32, ctypes.c_double,
                              ctypes.c_void_p)
    lib.ibp_status_string.argtypes = [i32]
    lib.ibp_status_string.restype = ctypes.c_char_p
    lib.ibp_slot_bytes.argtypes = [i64, i32, ctypes.POINTER(i64)]
    lib.ibp_meta_scratch_bytes.argtypes = [ctypes.POINTER(ctypes.c_size_t)]
    lib.ibp_build_meta.argtypes = [vp, i64, i64, i32, dbl, u32, vp, vp, vp]
    lib.ibp_compress.argtypes = [vp, i64, i64, i32, u32, vp, vp, i64, vp, vp, vp, vp]
    lib.ibp_decompress_gather.argtypes = [vp, i64, i64, i64, i32, u32, vp, vp, vp, i64, vp, vp, vp]
    lib.ibp_query.argtypes = [vp, vp, i64, i64, i32, vp, vp]
    lib.ibp_query_async.argtypes = [vp, vp, i64, i64, i32, vp, vp]
    lib.ibp_probe_read.argtypes = [vp, i64, vp, vp]
    lib.ibp_build_meta_noalloc.argtypes = [vp, i64, i64, i32, dbl, u32, vp, vp]
    lib.ibp_meta_select_scratch_bytes.argtypes = [ctypes.POINTER(ctypes.c_size_t)]
    lib.ibp_build_meta_select.argtypes = [vp, i64, i64, i32, dbl, u32, vp, vp, vp, vp]
    u64 = ctypes.c_uint64
    lib.ibp_meta_positions_scratch_bytes.argtypes = [i64, i32, ctypes.POINTER(ctypes.c_size_t)]
    lib.ibp_build_meta_positions.argtypes = [vp, i64, i64, i32, dbl, u32, vp, vp, vp, vp]
    lib.ibp_compress_positions.argtypes = [vp, i64, i64, i32, u32, vp, vp, vp, i64, vp, vp, vp]
    lib.ibp_decompress_gather_positions.argtypes = [vp, i64, i64, i64, i32, u32, vp, vp, vp, vp,
                                                    i64, vp, vp, vp]
    lib.ibp_meta_count.argtypes = [vp, i64, i64, i32, vp, vp]
    lib.ibp_gather_dedup_scratch_bytes.argtypes = [i64, i64, i32, u32, ctypes.POINTER(ctypes.c_size_t)]
    lib.ibp_decompress_gather_dedup.argtypes = [vp, i64, i64, i64, i32, u32, vp, vp, vp, i64, vp, vp,
                                                ctypes.c_size_t, vp, vp]
    lib.ibp_build_meta_block_positions.argtypes = [vp, i64, i64, i32, dbl, u32, vp, vp, vp, vp]
    lib.ibp_meta_finalize.argtypes = [vp, i64, i32, dbl, u32, vp, vp, vp]
    lib.ibp_decompress_gather_batched.argtypes = [vp, i32, i64, i32, u32, vp, vp]
    lib.ibp_decompress_gather_sized.argtypes = [vp, i64, i64, i64, i32, u32, vp, vp, vp, vp, i64,
                                                vp, vp, vp]
    lib.ibp_decompress_range.argtypes = [vp, i64, i64, i64, i32, u32, vp, vp, i64, i64, vp, vp, vp]
    lib.ibp_pack_scratch_bytes.argtypes = [i64, ctypes.POINTER(ctypes.c_size_t)]
    lib.ibp_pack_offsets.argtypes = [vp, vp, i64, i64, i32, vp, i64, vp, vp, vp, vp]
    lib.ibp_pack.argtypes = [vp, i64, i64, i64, i32, vp, vp, vp, i64, vp, vp, u64, vp, vp, vp, vp]
    lib.ibp_decompress_gather_packed.argtypes = [vp, u64, vp, i64, i64, i32, u32, vp, vp, vp, i64,
                                                 vp, vp, vp]
    szp = ctypes.POINTER(ctypes.c_size_t)
    lib.ibp_kv_append.argtypes = [vp, vp, vp, vp, vp]
    lib.ibp_kv_read.argtypes = [vp, vp, i64, vp, vp, i32, vp, vp]
    lib.ibp_kv_attention_scratch_bytes.argtypes = [vp, i64, i64, i32, i32, szp]
    lib.ibp_kv_attention.argtypes = [vp, vp, vp, ctypes.c_size_t, vp, vp]
    lib.ibp_kv_evict_scratch_bytes.argtypes = [vp, i64, szp]
    lib.ibp_kv_evict.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp, i64, vp, vp, ctypes.c_size_t,
                                 vp, vp]
    lib.ibp_kv_append_rotated.argtypes = [vp, vp, vp, vp, vp, vp, vp]
    lib.ibp_kv_bounds.argtypes = [vp, vp, vp, vp, vp]
    lib.ibp_kv_select_scratch_bytes.argtypes = [vp, szp]
    lib.ibp_kv_select.argtypes = [vp, vp, vp, i64, vp, vp, ctypes.c_size_t, vp, vp]
    lib.ibp_kv_attention_shared_scratch_bytes.argtypes = [vp, i64, i64, i32, i64, i64, szp]
    lib.ibp_kv_attention_shared.argtypes = [vp, vp, vp, vp, i64, i64, vp, ctypes.c_size_t, vp, vp]
    lib.ibp_kv_attention_selected_scratch_bytes.argtypes = [vp, i64, i64, i32, i64, szp]
    lib.ibp_kv_attention_selected.argtypes = [vp, vp, vp, i64, vp, ctypes.c_size_t, vp, vp]
    for name in SYMBOLS[1:]:
        getattr(lib, name).restype = i32
    lib.ibp_testing_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.ibp_testing_set_wait_limit_ns.restype = ctypes.c_uint64
    lib.ibp_testing_withhold_plans.argtypes = [ctypes.c_int]
    lib.ibp_testing_withhold_plans.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(code: int) -> str:
    try:
        return load().ibp_status_string(int(code)).decode()
    except RuntimeError:
        return "library not loaded"


def _check(rc: int, call: str) -> None:
    if rc != OK:
        raise IBPError(rc, call)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def dtype_code(t: torch.Tensor, dtype: int | None = None) -> int:
    if dtype is not None:
        return int(dtype)
    if t.dtype not in _TORCH_DTYPES:
        raise ValueError(f"pass dtype= for element tensors of {t.dtype}")
    return _TORCH_DTYPES[t.dtype]


def slot_bytes(row_elems: int, dtype: int) -> int:
    out = ctypes.c_int64(0)
    _check(load().ibp_slot_bytes(int(row_elems), int(dtype), ctypes.byref(out)), "ibp_slot_bytes")
    return out.value


def meta_scratch_bytes() -> int:
    out = ctypes.c_size_t(0)
    _check(load().ibp_meta_scratch_bytes(ctypes.byref(out)), "ibp_meta_scratch_bytes")
    return out.value


def _rows_shape(rows: torch.Tensor) -> tuple[int, int]:
    if rows.dim() != 2 or not rows.is_contiguous():
        raise ValueError("rows must be a contiguous 2-D tensor [n_rows, row_elems]")
    return rows.shape[0], rows.shape[1]


def build_meta(rows: torch.Tensor, T: float, block_elems: int, meta: torch.Tensor,
               scratch: torch.Tensor, dtype: int | None = None, stream=None) -> None:
    """ibp_build_meta: mask/bitval of ``rows`` into ``meta`` (16 device bytes)."""
    n, L = _rows_shape(rows)
    _check(load().ibp_build_meta(_ptr(rows), n, L, dtype_code(rows, dtype), float(T),
                                 int(block_elems), _ptr(meta), _ptr(scratch), _stream(stream)),
           "ibp_build_meta")


def meta_count(rows: torch.Tensor, counters: torch.Tensor, dtype: int | None = None,
               stream=None) -> None:
    """ibp_meta_count: per-bit 1-counts of ``rows`` into ``counters`` (32 x int64 on
    the device, overwritten); counters of several row sets add up."""
    n, L = _rows_shape(rows)
    _check(load().ibp_meta_count(_ptr(rows), n, L, dtype_code(rows, dtype), _ptr(counters),
                                 _stream(stream)), "ibp_meta_count")


def meta_finalize(counters: torch.Tensor, n_elems: int, dtype: int, T: float, block_elems: int,
                  meta: torch.Tensor, status: torch.Tensor | None = None, stream=None) -> None:
    """ibp_meta_finalize: the threshold rule applied to (summed) ``counters``; counters
    larger than ``n_elems`` give invalid metadata and ERR_META in ``status``."""
    _check(load().ibp_meta_finalize(_ptr(counters), int(n_elems), int(dtype), float(T),
                                    int(block_elems), _ptr(meta), _ptr(status),
                                    _stream(stream)),
           "ibp_meta_finalize")


def build_meta_noalloc(rows: torch.Tensor, T: float, block_elems: int, meta: torch.Tensor,
                       dtype: int | None = None, stream=None) -> None:
    """ibp_build_meta_noalloc: as build_meta, with the library's built-in counter
    array instead of caller scratch (for callers that cannot allocate)."""
    n, L = _rows_shape(rows)
    _check(load().ibp_build_meta_noalloc(_ptr(rows), n, L, dtype_code(rows, dtype), float(T),
                                         int(block_elems), _ptr(meta), _stream(stream)),
           "ibp_build_meta_noalloc")


def meta_select_scratch_bytes() -> int:
    out = ctypes.c_size_t(0)
    _check(load().ibp_meta_select_scratch_bytes(ctypes.byref(out)),
           "ibp_meta_select_scratch_bytes")
    return out.value


def build_meta_select(rows: torch.Tensor, T: float, block_elems: int, meta: torch.Tensor,
                      scratch: torch.Tensor, candidates: torch.Tensor | None = None,
                      dtype: int | None = None, stream=None) -> None:
    """ibp_build_meta_select: the saving-aware mask (the cheapest of the threshold
    mask and its nested reductions) into ``meta``; ``candidates`` (optional,
    MAX_MASK_CANDIDATES x 16 device bytes) receives every candidate and its score."""
    n, L = _rows_shape(rows)
    _check(load().ibp_build_meta_select(_ptr(rows), n, L, dtype_code(rows, dtype), float(T),
                                        int(block_elems), _ptr(meta), _ptr(candidates),
                                        _ptr(scratch), _stream(stream)), "ibp_build_meta_select")


def read_candidates(candidates: torch.Tensor) -> list[tuple[int, int, int]]:
    """(mask, bitval, stored_bytes) of every used entry of a candidate table."""
    raw = candidates.detach().to("cpu").contiguous().view(torch.uint8).numpy().tobytes()
    out = []
    for k in range(MAX_MASK_CANDIDATES):
        mask, bitval, stored = struct.unpack_from("<IIq", raw, 16 * k)
        if stored >= 0:
            out.append((mask, bitval, stored))
    return out


def compress(rows: torch.Tensor, block_elems: int, meta: torch.Tensor, slots: torch.Tensor,
             bitmask: torch.Tensor, row_bits: torch.Tensor | None = None,
             status: torch.Tensor | None = None, dtype: int | None = None,
             stream=None) -> None:
    """ibp_compress: encode ``rows`` into ``slots`` ([n_rows, slot_bytes] bytes)."""
    n, L = _rows_shape(rows)
    sb = slots.shape[1] * slots.element_size() if slots.dim() == 2 else slots.numel() * \
        slots.element_size() // max(n, 1)
    _check(load().ibp_compress(_ptr(rows), n, L, dtype_code(rows, dtype), int(block_elems),
                               _ptr(meta), _ptr(slots), sb, _ptr(bitmask), _ptr(row_bits),
                               _ptr(status), _stream(stream)), "ibp_compress")


def decompress_gather(slots: torch.Tensor, n_rows: int, row_elems: int, dtype: int,
                      block_elems: int, bitmask: torch.Tensor, meta: torch.Tensor,
                      idx: torch.Tensor, out: torch.Tensor, status: torch.Tensor | None = None,
                      stream=None) -> None:
    """ibp_decompress_gather: rows ``idx`` rebuilt into ``out`` [n_idx, row_elems]."""
    sb = slots.shape[1] * slots.element_size() if slots.dim() == 2 else slots.numel() * \
        slots.element_size() // max(int(n_rows), 1)
    if idx.dtype != torch.int64:
        raise ValueError("idx must be int64")
    _check(load().ibp_decompress_gather(_ptr(slots), sb, int(n_rows), int(row_elems), int(dtype),
                                        int(block_elems), _ptr(bitmask), _ptr(meta), _ptr(idx),
                                        idx.numel(), _ptr(out), _ptr(status), _stream(stream)),
           "ibp_decompress_gather")


def gather_dedup_scratch_bytes(n_idx: int, row_elems: int, dtype: int, block_elems: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().ibp_gather_dedup_scratch_bytes(int(n_idx), int(row_elems), int(dtype),
                                                 int(block_elems), ctypes.byref(out)),
           "ibp_gather_dedup_scratch_bytes")
    return out.value


def decompress_gather_dedup(slots: torch.Tensor, n_rows: int, row_elems: int, dtype: int,
                            block_elems: int, bitmask: torch.Tensor, meta: torch.Tensor,
                            idx: torch.Tensor, out: torch.Tensor, scratch: torch.Tensor,
                            status: torch.Tensor | None = None, stream=None) -> None:
    """ibp_decompress_gather_dedup: the result of decompress_gather, each distinct
    row read and decoded once (``scratch``: gather_dedup_scratch_bytes bytes)."""
    sb = slots.shape[1] * slots.element_size() if slots.dim() == 2 else slots.numel() * \
        slots.element_size() // max(int(n_rows), 1)
    if idx.dtype != torch.int64:
        raise ValueError("idx must be int64")
    _check(load().ibp_decompress_gather_dedup(
        _ptr(slots), sb, int(n_rows), int(row_elems), int(dtype), int(block_elems), _ptr(bitmask),
        _ptr(meta), _ptr(idx), idx.numel(), _ptr(out), _ptr(scratch),
        scratch.nbytes, _ptr(status), _stream(stream)),
        "ibp_decompress_gather_dedup")


def pack_scratch_bytes(n_sel: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().ibp_pack_scratch_bytes(int(n_sel), ctypes.byref(out)), "ibp_pack_scratch_bytes")
    return out.value


def pack_offsets(bitmask: torch.Tensor, row_bits: torch.Tensor, n_rows: int, row_elems: int,
                 dtype: int, offsets: torch.Tensor, scratch: torch.Tensor,
                 sel: torch.Tensor | None = None, n_sel: int | None = None,
                 status: torch.Tensor | None = None, stream=None) -> None:
    """ibp_pack_offsets: entry offsets ([n_sel + 1] int64 on the device) of a packed
    store of rows ``sel`` (all rows when None)."""
    if sel is not None and sel.dtype != torch.int64:
        raise ValueError("sel must be int64")
    ns = int(n_sel) if n_sel is not None else (sel.numel() if sel is not None else int(n_rows))
    _check(load().ibp_pack_offsets(_ptr(bitmask), _ptr(row_bits), int(n_rows), int(row_elems),
                                   int(dtype), _ptr(sel), ns, _ptr(offsets), _ptr(scratch),
                                   _ptr(status), _stream(stream)), "ibp_pack_offsets")


def pack(slots: torch.Tensor, n_rows: int, row_elems: int, dtype: int, bitmask: torch.Tensor,
         row_bits: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor,
         pack_bitmask: torch.Tensor, pack_row_bits: torch.Tensor | None = None,
         sel: torch.Tensor | None = None, n_sel: int | None = None,
         status: torch.Tensor | None = None, stream=None) -> None:
    """ibp_pack: copy the entries of a packed store into ``packed``."""
    sb = slots.shape[1] * slots.element_size() if slots.dim() == 2 else slots.numel() * \
        slots.element_size() // max(int(n_rows), 1)
    ns = int(n_sel) if n_sel is not None else (sel.numel() if sel is not None else int(n_rows))
    _check(load().ibp_pack(_ptr(slots), sb, int(n_rows), int(row_elems), int(dtype),
                           _ptr(bitmask), _ptr(row_bits), _ptr(sel), ns, _ptr(offsets),
                           _ptr(packed), packed.numel() * packed.element_size(),
                           _ptr(pack_bitmask), _ptr(pack_row_bits), _ptr(status),
                           _stream(stream)), "ibp_pack")


def decompress_gather_packed(packed: torch.Tensor, offsets: torch.Tensor, n_rows: int,
                             row_elems: int, dtype: int, block_elems: int, bitmask: torch.Tensor,
                             meta: torch.Tensor, idx: torch.Tensor, out: torch.Tensor,
                             status: torch.Tensor | None = None, stream=None) -> None:
    """ibp_decompress_gather_packed: rows ``idx`` of a packed store into ``out``."""
    if idx.dtype != torch.int64:
        raise ValueError("idx must be int64")
    _check(load().ibp_decompress_gather_packed(
        _ptr(packed), packed.numel() * packed.element_size(), _ptr(offsets), int(n_rows),
        int(row_elems), int(dtype), int(block_elems), _ptr(bitmask), _ptr(meta), _ptr(idx),
        idx.numel(), _ptr(out), _ptr(status), _stream(stream)), "ibp_decompress_gather_packed")


def meta_positions_scratch_bytes(row_elems: int, dtype: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().ibp_meta_positions_scratch_bytes(int(row_elems), int(dtype), ctypes.byref(out)),
           "ibp_meta_positions_scratch_bytes")
    return out.value


def build_meta_block_positions(rows: torch.Tensor, T: float, block_elems: int,
                               pmask: torch.Tensor, pbitval: torch.Tensor, scratch: torch.Tensor,
                               dtype: int | None = None, stream=None) -> None:
    """ibp_build_meta_block_positions: one mask/bitval per position within a block,
    written row-sized (entry e holds the pair of position e % block_elems)."""
    n, L = _rows_shape(rows)
    _check(load().ibp_build_meta_block_positions(_ptr(rows), n, L, dtype_code(rows, dtype),
                                                 float(T), int(block_elems), _ptr(pmask),
                                                 _ptr(pbitval), _ptr(scratch), _stream(stream)),
           "ibp_build_meta_block_positions")


def build_meta_positions(rows: torch.Tensor, T: float, block_elems: int, pmask: torch.Tensor,
                         pbitval: torch.Tensor, scratch: torch.Tensor, dtype: int | None = None,
                         stream=None) -> None:
    """ibp_build_meta_positions: one mask/bitval per element position of a row."""
    n, L = _rows_shape(rows)
    _check(load().ibp_build_meta_positions(_ptr(rows), n, L, dtype_code(rows, dtype), float(T),
                                           int(block_elems), _ptr(pmask), _ptr(pbitval),
                                           _ptr(scratch), _stream(stream)),
           "ibp_build_meta_positions")


def compress_positions(rows: torch.Tensor, block_elems: int, pmask: torch.Tensor,
                       pbitval: torch.Tensor, slots: torch.Tensor, bitmask: torch.Tensor,
                       row_bits: torch.Tensor | None = None, dtype: int | None = None,
                       stream=None) -> None:
    """ibp_compress_positions: encode ``rows`` with per-position metadata."""
    n, L = _rows_shape(rows)
    sb = slots.shape[1] * slots.element_size() if slots.dim() == 2 else slots.numel() * \
        slots.element_size() // max(n, 1)
    _check(load().ibp_compress_positions(_ptr(rows), n, L, dtype_code(rows, dtype),
                                         int(block_elems), _ptr(pmask), _ptr(pbitval),
                                         _ptr(slots), sb, _ptr(bitmask), _ptr(row_bits),
                                         _stream(stream)), "ibp_compress_positions")


def decompress_gather_positions(slots: torch.Tensor, n_rows: int, row_elems: int, dtype: int,
                                block_elems: int, bitmask: torch.Tensor, pmask: torch.Tensor,
                                pbitval: torch.Tensor, idx: torch.Tensor, out: torch.Tensor,
                                status: torch.Tensor | None = None, stream=None) -> None:
    """ibp_decompress_gather_positions: rows ``idx`` rebuilt with per-position metadata."""
    if idx.dtype != torch.int64:
        raise ValueError("idx must be int64")
    sb = slots.shape[1] * slots.element_size() if slots.dim() == 2 else slots.numel() * \
        slots.element_size() // max(int(n_rows), 1)
    _check(load().ibp_decompress_gather_positions(
        _ptr(slots), sb, int(n_rows), int(row_elems), int(dtype), int(block_elems),
        _ptr(bitmask), _ptr(pmask), _ptr(pbitval), _ptr(idx), idx.numel(), _ptr(out),
        _ptr(status), _stream(stream)), "ibp_decompress_gather_positions")


def decompress_gather_sized(slots: torch.Tensor, n_rows: int, row_elems: int, dtype: int,
                            block_elems: int, bitmask: torch.Tensor, row_bits: torch.Tensor,
                            meta: torch.Tensor, idx: torch.Tensor, out: torch.Tensor,
                            status: torch.Tensor | None = None, stream=None) -> None:
    """ibp_decompress_gather_sized: as decompress_gather, staging only each row's
    stored bytes (known from ``row_bits``)."""
    if idx.dtype != torch.int64:
        raise ValueError("idx must be int64")
    sb = slots.shape[1] * slots.element_size() if slots.dim() == 2 else slots.numel() * \
        slots.element_size() // max(int(n_rows), 1)
    _check(load().ibp_decompress_gather_sized(
        _ptr(slots), sb, int(n_rows), int(row_elems), int(dtype), int(block_elems),
        _ptr(bitmask), _ptr(row_bits), _ptr(meta), _ptr(idx), idx.numel(), _ptr(out),
        _ptr(status), _stream(stream)), "ibp_decompress_gather_sized")


def decompress_gather_batched(jobs, row_elems: int, dtype: int, block_elems: int,
                              status: torch.Tensor | None = None, stream=None) -> None:
    """ibp_decompress_gather_batched: ``jobs`` is a list of (slots, n_rows, bitmask, meta,
    idx, out) tuples sharing one row geometry; one launch per 64 jobs."""
    arr = (GatherJob * max(len(jobs), 1))()
    for k, (slots, n_rows, bitmask, meta, idx, out) in enumerate(jobs):
        if idx.dtype != torch.int64:
            raise ValueError("idx must be int64")
        sb = slots.shape[1] * slots.element_size() if slots.dim() == 2 else slots.numel() * \
            slots.element_size() // max(int(n_rows), 1)
        arr[k] = GatherJob(slots.data_ptr(), sb, int(n_rows), bitmask.data_ptr(), meta.data_ptr(),
                           idx.data_ptr(), idx.numel(), out.data_ptr())
    _check(load().ibp_decompress_gather_batched(ctypes.cast(arr, ctypes.c_void_p), len(jobs),
                                                int(row_elems), int(dtype), int(block_elems),
                                                _ptr(status), _stream(stream)),
           "ibp_decompress_gather_batched")


def decompress_range(slots: torch.Tensor, n_rows: int, row_elems: int, dtype: int,
                     block_elems: int, bitmask: torch.Tensor, meta: torch.Tensor, row_begin: int,
                     n_out: int, out: torch.Tensor, status: torch.Tensor | None = None,
                     stream=None) -> None:
    """ibp_decompress_range: rows row_begin .. row_begin + n_out - 1 into ``out``."""
    sb = slots.shape[1] * slots.element_size() if slots.dim() == 2 else slots.numel() * \
        slots.element_size() // max(int(n_rows), 1)
    _check(load().ibp_decompress_range(_ptr(slots), sb, int(n_rows), int(row_elems), int(dtype),
                                       int(block_elems), _ptr(bitmask), _ptr(meta),
                                       int(row_begin), int(n_out), _ptr(out), _ptr(status),
                                       _stream(stream)), "ibp_decompress_range")


def query(bitmask: torch.Tensor, row_bits: torch.Tensor, n_rows: int, row_elems: int, dtype: int,
          stream=None) -> Stats:
    """ibp_query: store statistics, returned in host memory (synchronises the stream)."""
    out = Stats()
    _check(load().ibp_query(_ptr(bitmask), _ptr(row_bits), int(n_rows), int(row_elems),
                            int(dtype), ctypes.byref(out), _stream(stream)), "ibp_query")
    return out


def query_async(bitmask: torch.Tensor, row_bits: torch.Tensor, n_rows: int, row_elems: int,
                dtype: int, stats: torch.Tensor, stream=None) -> None:
    """ibp_query_async: store statistics into ``stats`` (40 device bytes, see Stats),
    asynchronously."""
    _check(load().ibp_query_async(_ptr(bitmask), _ptr(row_bits), int(n_rows), int(row_elems),
                                  int(dtype), _ptr(stats), _stream(stream)), "ibp_query_async")


def read_stats(stats: torch.Tensor) -> Stats:
    host = stats.detach().to("cpu").contiguous().view(torch.uint8).numpy().tobytes()
    return Stats.from_buffer_copy(host[:ctypes.sizeof(Stats)])


_KV_CODES = {torch.int8: KV_INT8}
if hasattr(torch, "float8_e4m3fn"):
    _KV_CODES[torch.float8_e4m3fn] = KV_E4M3


def _at(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream):
    # the current stream's handle without building a Stream object around it
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) if stream is None \
        else stream.cuda_stream


class KVCache:
    """Handle of an 8-bit paged key/value cache (``ibp_kv_cache``): the tensors it is
    made of, which the caller owns and keeps where they are.

    k_codes, v_codes: [n_pages, n_heads, page_tokens, head_dim], int8 or float8_e4m3fn;
    k_scales, v_scales: [n_pages, n_heads] float32; table: [batch, columns] int32 page ids
    (unused entries are not read); lens: [batch] int32 tokens held. page_tokens is 16, 32,
    64 or 128, head_dim 64 or 128. Several handles may share the page pools."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scales: torch.Tensor,
                 v_scales: torch.Tensor, table: torch.Tensor, lens: torch.Tensor):
        if k_codes.dim() != 4 or k_codes.shape != v_codes.shape or \
                k_codes.dtype != v_codes.dtype or k_codes.dtype not in _KV_CODES:
            raise ValueError("k_codes and v_codes must be int8 or float8_e4m3fn tensors "
                             "[n_pages, n_heads, page_tokens, head_dim]")
        if any(s.shape != k_codes.shape[:2] or s.dtype != torch.float32
               for s in (k_scales, v_scales)):
            raise ValueError("k_scales and v_scales must be float32 [n_pages, n_heads]")
        if table.dim() != 2 or table.dtype != torch.int32 or \
                (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("table must be int32 [batch, columns], its rows contiguous")
        if lens.dtype != torch.int32 or lens.shape != table.shape[:1]:
            raise ValueError("lens must be int32 [batch]")
        for t in (k_codes, v_codes, k_scales, v_scales, lens):
            if not t.is_contiguous():
                raise ValueError("codes, scales and lens must be contiguous")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, \
            v_scales
        self.table, self.lens = table, lens
        n, h, p, d = k_codes.shape
        stride = table.stride(0) if table.shape[0] > 1 else table.shape[1]
        self.batch, self.n_heads, self.page_tokens, self.head_dim = table.shape[0], h, p, d
        self.capacity = table.shape[1] * p
        self.bounds_shape = (n, h, 2, d)
        self.struct = KVCacheStruct(_at(k_codes), _at(v_codes), _at(k_scales), _at(v_scales),
                                    _at(table), _at(lens), n, stride, table.shape[0],
                                    table.shape[1], h, p, d, _KV_CODES[k_codes.dtype])
        self.address = ctypes.addressof(self.struct)


def _head_rows(t: torch.Tensor, cache: KVCache, heads: int, what: str) -> tuple[int, int]:
    """Row and head strides of [n_rows, heads, head_dim] rows (elements of a head contiguous)."""
    shape, strides, d = t.shape, t.stride(), cache.head_dim
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or (strides[2] != 1 and t.numel()):
        raise ValueError(f"{what} must be [n_rows, {heads}, {d}] with the elements of a head "
                         "contiguous")
    n = shape[0]
    return strides[0] if n > 1 else heads * d, strides[1] if n and heads > 1 else d


def _int32(t: torch.Tensor | None, n: int, what: str):
    if t is not None and (t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous int32 tensor of {n} entries")
    return _at(t)


def rotation_table(n_positions: int, dim: int, base: float = 10000.0,
                   device: torch.device | str = "cuda") -> torch.Tensor:
    """Cosines and sines [n_positions, dim/2, 2] of the angles p * base^(-2i/dim), which are
    taken in 64 bits (in 32 those of far positions are off by whole fractions of a turn)."""
    pairs = dim // 2
    inverse = float(base) ** (-torch.arange(pairs, dtype=torch.float64, device=device) / pairs)
    out = torch.empty((n_positions, pairs, 2), dtype=torch.float32, device=device)
    for at in range(0, n_positions, 1 << 16):  # 64-bit angles of a part at a time
        p = torch.arange(at, min(at + (1 << 16), n_positions), dtype=torch.float64, device=device)
        angle = p[:, None] * inverse[None, :]
        out[at:at + p.numel(), :, 0] = angle.cos()
        out[at:at + p.numel(), :, 1] = angle.sin()
    return out


class KVRotation:
    """Rotation of positions (``ibp_kv_rotation``): ``table`` [n_positions, dim/2, 2] float32,
    the cosine and sine of each pair at each position (``rotation_table``, or a caller's own
    scaling of the angles); ``axis``: the axis of positions that each pair goes by, numbers
    from 0 to 3 (None: one axis); ``interleaved``: pairs are (2i, 2i + 1) instead of
    (i, i + dim/2). The caller keeps the table where it is."""

    def __init__(self, table: torch.Tensor, axis=None, interleaved: bool = False):
        if table.dim() != 3 or table.shape[2] != 2 or table.dtype != torch.float32 or \
                not table.is_contiguous():
            raise ValueError("table must be contiguous float32 [n_positions, dim/2, 2]")
        pairs = table.shape[1]
        axis = [0] * pairs if axis is None else [int(a) for a in axis]
        if len(axis) != pairs or pairs > 64 or any(not 0 <= a < 4 for a in axis):
            raise ValueError(f"axis must be {pairs} numbers from 0 to 3, of 64 pairs at most")
        self.table, self.axes = table, max(axis, default=0) + 1
        self.struct = KVRotationStruct(_at(table), None, table.shape[0], 2 * pairs, self.axes,
                                       int(bool(interleaved)), (ctypes.c_uint8 * 64)(*axis))


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor | None = None,
              new_lens: torch.Tensor | None = None, status: torch.Tensor | None = None,
              stream=None) -> None:
    """ibp_kv_append: quantise rows ``k`` and ``v`` ([n_rows, n_heads, head_dim]; sequence
    b owns rows cu[b]..cu[b+1]-1, or n_rows/batch each) into the pages behind
    ``cache.lens``; ``new_lens`` receives the lengths after the call."""
    kr, kh = _head_rows(k, cache, cache.n_heads, "k")
    vr, vh = _head_rows(v, cache, cache.n_heads, "v")
    if v.dtype != k.dtype or v.shape[0] != k.shape[0]:
        raise ValueError("k and v must have one dtype and row count")
    rows = KVRows(_at(k), _at(v), _int32(cu, cache.batch + 1, "cu"), k.shape[0], kr, kh, vr, vh,
                  dtype_code(k))
    _check(load().ibp_kv_append(cache.address, ctypes.addressof(rows),
                                _int32(new_lens, cache.batch, "new_lens"), _at(status),
                                _raw_stream(stream)), "ibp_kv_append")


def kv_append_rotated(cache: KVCache, k: torch.Tensor, v: torch.Tensor, rotation: KVRotation,
                      positions: torch.Tensor | None = None, q: torch.Tensor | None = None,
                      q_out: torch.Tensor | None = None, cu: torch.Tensor | None = None,
                      new_lens: torch.Tensor | None = None, status: torch.Tensor | None = None,
                      stream=None) -> None:
    """ibp_kv_append_rotated: ``kv_append`` with ``rotation`` applied to ``k`` on the way, and
    to the query rows ``q`` ([n_rows, q_heads, head_dim], k's type), which go to ``q_out``
    (None: q itself). ``positions``: int32 [n_rows, axes] (None: each row's place in the cache,
    which after an eviction is not its token's number any more)."""
    kr, kh = _head_rows(k, cache, cache.n_heads, "k")
    vr, vh = _head_rows(v, cache, cache.n_heads, "v")
    n = k.shape[0]
    dtype = k.dtype
    if v.dtype != dtype or v.shape[0] != n:
        raise ValueError("k and v must have one dtype and row count")
    rows = KVRows(_at(k), _at(v), _int32(cu, cache.batch + 1, "cu"), n, kr, kh, vr, vh,
                  dtype_code(k))
    turn = KVRotationStruct.from_buffer_copy(rotation.struct)
    turn.d_positions = _int32(positions, n * rotation.axes, "positions")
    queries = None
    if q is not None:
        shape = q.shape
        if q_out is None:
            q_out = q
        elif q_out.dtype != dtype or q_out.shape != shape:
            raise ValueError("q_out must have q's dtype and shape")
        if q.dtype != dtype or shape[0] != n:
            raise ValueError("q must have k's dtype and row count")
        heads = shape[1] if len(shape) == 3 else 0
        qr, qh = _head_rows(q, cache, heads, "q")
        orow, oh = (qr, qh) if q_out is q else _head_rows(q_out, cache, heads, "q_out")
        queries = KVTurned(_at(q), _at(q_out), qr, qh, orow, oh, heads)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _check(load().ibp_kv_append_rotated(
        cache.address, ctypes.addressof(rows), ctypes.addressof(turn),
        None if queries is None else ctypes.addressof(queries),
        _int32(new_lens, cache.batch, "new_lens"), _at(status), _raw_stream(stream)),
        "ibp_kv_append_rotated")


def kv_read(cache: KVCache, k_out: torch.Tensor | None, v_out: torch.Tensor | None,
            begin: torch.Tensor | None = None, status: torch.Tensor | None = None,
            stream=None) -> None:
    """ibp_kv_read: tokens begin[b] (0 when None) and on of every sequence as values into
    ``k_out`` and ``v_out`` ([batch, n_out, n_heads, head_dim], either may be None); zeros
    past the length."""
    given = [t for t in (k_out, v_out) if t is not None]
    if not given:
        return
    for t in given:
        if t.dim() != 4 or not t.is_contiguous() or t.dtype != given[0].dtype or \
                t.shape != (cache.batch, given[0].shape[1], cache.n_heads, cache.head_dim):
            raise ValueError("k_out and v_out must be contiguous [batch, n_out, n_heads, "
                             "head_dim] tensors of one dtype")
    _check(load().ibp_kv_read(cache.address, _int32(begin, cache.batch, "begin"),
                              given[0].shape[1], _at(k_out), _at(v_out), dtype_code(given[0]),
                              _at(status), _raw_stream(stream)), "ibp_kv_read")


def _query(cache: KVCache, q: torch.Tensor, out: torch.Tensor | None, scale: float, cu_q, max_q,
           lse) -> KVQuery:
    """ibp_kv_query of query rows, without weights. (It is on the path of every decoding step:
    each attribute of a tensor is asked for once.)"""
    shape, dtype = q.shape, q.dtype
    heads = shape[1] if len(shape) == 3 else 0
    qr, qh = _head_rows(q, cache, heads, "q")
    n = shape[0]
    out_at = lse_at = None
    orow = oh = 0
    if out is not None:
        if out.dtype != dtype or out.shape != shape:
            raise ValueError("out must have q's dtype and shape")
        orow, oh = _head_rows(out, cache, heads, "out")
        out_at = out.data_ptr()
    if lse is not None:
        if lse.dtype != torch.float32 or lse.numel() != n * heads or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous float32 tensor [n_rows, q_heads]")
        lse_at = lse.data_ptr()
    if max_q is None:
        if cu_q is not None:
            raise ValueError("cu_q needs max_q, the most rows that a sequence has")
        max_q = n // max(cache.batch, 1)
    return KVQuery(q.data_ptr(), out_at, lse_at,
                   None if cu_q is None else _int32(cu_q, cache.batch + 1, "cu_q"), None, None, n,
                   max_q, 0, qr, qh, orow, oh, heads,
                   _TORCH_DTYPES[dtype] if dtype in _TORCH_DTYPES else dtype_code(q), scale, 1.0)


def _bounds(cache: KVCache, bounds: torch.Tensor):
    if bounds.dtype != torch.int8 or bounds.shape != cache.bounds_shape or \
            not bounds.is_contiguous():
        raise ValueError(f"bounds must be contiguous int8 {list(cache.bounds_shape)}")
    return bounds.data_ptr()


def _columns(cache: KVCache, columns: torch.Tensor) -> int:
    """How many columns the lists hold."""
    shape = columns.shape
    if len(shape) != 3 or shape[0] != cache.batch or shape[1] != cache.n_heads or \
            columns.dtype != torch.int32 or not columns.is_contiguous():
        raise ValueError("columns must be contiguous int32 [batch, n_heads, pages]")
    return shape[2]


def kv_attention_scratch_bytes(cache: KVCache, n_rows: int, max_q: int, q_heads: int,
                               with_weights: bool) -> int:
    out = ctypes.c_size_t(0)
    _check(load().ibp_kv_attention_scratch_bytes(cache.address, int(n_rows), int(max_q),
                                                 int(q_heads), int(bool(with_weights)),
                                                 ctypes.byref(out)),
           "ibp_kv_attention_scratch_bytes")
    return out.value


def kv_attention(cache: KVCache, q: torch.Tensor, out: torch.Tensor, scale: float,
                 scratch: torch.Tensor, cu_q: torch.Tensor | None = None,
                 max_q: int | None = None, lse: torch.Tensor | None = None,
                 weights: torch.Tensor | None = None, weights_in: torch.Tensor | None = None,
                 decay: float = 1.0, status: torch.Tensor | None = None, stream=None) -> None:
    """ibp_kv_attention: softmax(scale * q k) v of the query rows ``q`` ([n_rows, q_heads,
    head_dim], float16 or bfloat16; sequence b owns rows cu_q[b]..cu_q[b+1]-1, at most
    ``max_q`` of them, the last of which stands at its last token) into ``out``; ``lse``
    [n_rows, q_heads] float32; ``weights`` [batch, n_heads, >= capacity] float32 receives
    decay * weights_in + the probabilities summed over rows and shared heads."""
    n, heads = q.shape[0], q.shape[1]
    stride = 0
    if weights is not None:
        stride = weights.shape[-1]
        for t in (weights, weights_in):
            if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or
                                  t.shape != (cache.batch, cache.n_heads, stride)):
                raise ValueError("weights must be contiguous float32 [batch, n_heads, stride]")
    query = _query(cache, q, out, scale, cu_q, max_q, lse)
    query.d_weights_in, query.d_weights = _at(weights_in), _at(weights)
    query.weights_stride, query.decay = stride, decay
    _check(load().ibp_kv_attention(cache.address, ctypes.addressof(query), _at(scratch),
                                   scratch.nbytes, _at(status),
                                   _raw_stream(stream)), "ibp_kv_attention")


def kv_bounds(cache: KVCache, bounds: torch.Tensor, begin: torch.Tensor | None = None,
              status: torch.Tensor | None = None, stream=None) -> None:
    """ibp_kv_bounds: least and largest K code of each element over a page's tokens into
    ``bounds`` (int8 [n_pages, n_heads, 2, head_dim]), for the pages of tokens begin[b] (0 when
    None) and on of every sequence."""
    _check(load().ibp_kv_bounds(cache.address, _bounds(cache, bounds),
                                _int32(begin, cache.batch, "begin"), _at(status),
                                _raw_stream(stream)), "ibp_kv_bounds")


def kv_select_scratch_bytes(cache: KVCache) -> int:
    out = ctypes.c_size_t(0)
    _check(load().ibp_kv_select_scratch_bytes(cache.address, ctypes.byref(out)),
           "ibp_kv_select_scratch_bytes")
    return out.value


def kv_select(cache: KVCache, bounds: torch.Tensor, q: torch.Tensor, columns: torch.Tensor,
              scratch: torch.Tensor, cu_q: torch.Tensor | None = None, max_q: int | None = None,
              status: torch.Tensor | None = None, stream=None) -> None:
    """ibp_kv_select: the pages of every sequence and K/V head that the query rows ``q`` (as in
    ``kv_attention``) score highest by ``bounds``, the first page and the rows' own among them,
    as columns of the page table into ``columns`` (int32 [batch, n_heads, pages], rising, then
    -1)."""
    query = _query(cache, q, None, 1.0, cu_q, max_q, None)
    _check(load().ibp_kv_select(cache.address, _bounds(cache, bounds), ctypes.addressof(query),
                                _columns(cache, columns), _at(columns), _at(scratch),
                                scratch.nbytes, _at(status),
                                _raw_stream(stream)), "ibp_kv_select")


def kv_attention_selected_scratch_bytes(cache: KVCache, n_rows: int, max_q: int, q_heads: int,
                                        pages: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().ibp_kv_attention_selected_scratch_bytes(cache.address, int(n_rows), int(max_q),
                                                          int(q_heads), int(pages),
                                                          ctypes.byref(out)),
           "ibp_kv_attention_selected_scratch_bytes")
    return out.value


def kv_attention_selected(cache: KVCache, columns: torch.Tensor, q: torch.Tensor,
                          out: torch.Tensor, scale: float, scratch: torch.Tensor,
                          cu_q: torch.Tensor | None = None, max_q: int | None = None,
                          lse: torch.Tensor | None = None, status: torch.Tensor | None = None,
                          stream=None) -> None:
    """ibp_kv_attention_selected: ``kv_attention`` over the pages that ``columns`` (as
    ``kv_select`` writes it) names."""
    query = _query(cache, q, out, scale, cu_q, max_q, lse)
    _check(load().ibp_kv_attention_selected(cache.address, ctypes.addressof(query), _at(columns),
                                            _columns(cache, columns), _at(scratch),
                                            scratch.nbytes, _at(status),
                                            _raw_stream(stream)), "ibp_kv_attention_selected")


def kv_attention_shared_scratch_bytes(cache: KVCache, n_rows: int, max_q: int, q_heads: int,
                                      n_groups: int, group_rows: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().ibp_kv_attention_shared_scratch_bytes(cache.address, int(n_rows), int(max_q),
                                                        int(q_heads), int(n_groups),
                                                        int(group_rows), ctypes.byref(out)),
           "ibp_kv_attention_shared_scratch_bytes")
    return out.value


def kv_attention_shared(cache: KVCache, q: torch.Tensor, out: torch.Tensor, scale: float,
                        scratch: torch.Tensor, groups: torch.Tensor, prefix: torch.Tensor,
                        group_rows: int, cu_q: torch.Tensor | None = None,
                        max_q: int | None = None, lse: torch.Tensor | None = None,
                        status: torch.Tensor | None = None, stream=None) -> None:
    """ibp_kv_attention_shared: ``kv_attention`` where the sequences groups[g]..groups[g+1]-1
    (int32 [n_groups + 1]) share their first prefix[g] tokens (int32 [n_groups]) and the pages
    of these, each beginning gone over once for the whole group; ``group_rows``: the most
    query rows of one group."""
    query = _query(cache, q, out, scale, cu_q, max_q, lse)
    n = prefix.numel()
    _check(load().ibp_kv_attention_shared(
        cache.address, ctypes.addressof(query), _int32(groups, n + 1, "groups"),
        _int32(prefix, n, "prefix"), n, int(group_rows), _at(scratch),
        scratch.nbytes, _at(status), _raw_stream(stream)),
        "ibp_kv_attention_shared")


def kv_evict_scratch_bytes(cache: KVCache, budget: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().ibp_kv_evict_scratch_bytes(cache.address, int(budget), ctypes.byref(out)),
           "ibp_kv_evict_scratch_bytes")
    return out.value


def kv_evict(cache: KVCache, weights: torch.Tensor, budget: int, recent: int, dst: KVCache,
             scratch: torch.Tensor, new_weights: torch.Tensor | None = None,
             kept: torch.Tensor | None = None, status: torch.Tensor | None = None,
             stream=None) -> None:
    """ibp_kv_evict: the last ``recent`` tokens and the budget - recent of the largest
    ``weights`` ([batch, n_heads, >= capacity] float32) of every longer sequence and head,
    requantised into ``dst``'s pages; ``dst.lens`` receives the new lengths,
    ``new_weights`` ([batch, n_heads, >= budget]) and ``kept`` ([batch, n_heads, budget]
    int32) the kept tokens' weights and old positions."""
    for t in (weights, new_weights):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or t.dim() != 3 or
                              t.shape[:2] != (cache.batch, cache.n_heads)):
            raise ValueError("weights must be contiguous float32 [batch, n_heads, stride]")
    _check(load().ibp_kv_evict(
        cache.address, _at(weights), weights.shape[2], int(budget), int(recent), dst.address,
        _at(dst.lens), _at(new_weights), 0 if new_weights is None else new_weights.shape[2],
        _int32(kept, cache.batch * cache.n_heads * int(budget), "kept"), _at(scratch),
        scratch.nbytes, _at(status), _raw_stream(stream)),
        "ibp_kv_evict")


def probe_read(src: torch.Tensor, sink: torch.Tensor, nbytes: int | None = None,
               stream=None) -> None:
    """ibp_probe_read: stream ``nbytes`` of ``src`` through the GPU (bandwidth probe)."""
    n = src.numel() * src.element_size() if nbytes is None else int(nbytes)
    _check(load().ibp_probe_read(_ptr(src), n, _ptr(sink), _stream(stream)), "ibp_probe_read")


def testing_set_wait_limit_ns(ns: int) -> int:
    """ibp_testing_set_wait_limit_ns (include/ibp_testing.h): the limit of the gather
    and attention kernels' bounded waits, in ns (0: the default 2 s); returns the previous one."""
    return int(load().ibp_testing_set_wait_limit_ns(int(ns)))


def testing_withhold_plans(on: bool) -> bool:
    """ibp_testing_withhold_plans (include/ibp_testing.h): the warp-specialised
    gather's planners keep their plans from the decoders, the attention kernels' fetching
    warps stop early; returns the previous setting."""
    return bool(load().ibp_testing_withhold_plans(1 if on else 0))
