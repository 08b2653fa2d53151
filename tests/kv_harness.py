"""Shared set-up of the key/value cache tests: random rows, a reference cache, and the
same cache as page pools whose unused slots and pages hold what must never be used."""
from __future__ import annotations

import numpy as np
import torch

import lossless_bit_level_gb300 as ibp
import kv_reference as ref

TORCH_CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def rounded(x: np.ndarray, dtype: str) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(DTYPES[dtype])


def random_rows(rng, n, heads, dim, dtype="bf16", spread=True):
    """{"k", "v"}: torch tensors [n, heads, dim]; a few channels ten times as large."""
    out = {}
    for name in "kv":
        x = rng.standard_normal((n, heads, dim)).astype(np.float32)
        if spread and n:
            x[:, :, rng.integers(0, dim)] *= 10
        out[name] = rounded(x, dtype)
    return out


def as_float32(rows):
    return {n: t.float().numpy() for n, t in rows.items()}


def code_bytes(c: np.ndarray, code: str) -> np.ndarray:
    if code == "int8":
        return c.astype(np.int8).view(np.uint8)
    return torch.from_numpy(c.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def pools(cache: ref.Cache, rng, room=0, cols=None, spare=2, device="cuda"):
    """ibp.KVCache of the reference cache (on the GPU): pages in random order, `room`
    tokens of pages past every length, stale slots and pages full of NaN codes (e4m3) or
    -128 (int8) and NaN scales, unused table entries -1."""
    P, H, D = cache.page, cache.heads, cache.dim
    need = [-(-(n + room) // P) for n in cache.lens]
    n_pages = sum(need) + spare
    cols = max(cols or 0, max(need, default=0), 1)
    order = rng.permutation(n_pages)
    table = np.full((cache.batch, cols), -1, np.int32)
    stale = 0x80 if cache.code == "int8" else 0x7F
    at, got = 0, {}
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    for name in "kv":
        codes = np.full((n_pages, H, P, D), stale, np.uint8)
        scales = np.full((n_pages, H), np.nan, np.float32)
        for b in range(cache.batch):
            for h in range(H):
                for j, (s, c) in enumerate(cache.tiles[name][b][h]):
                    codes[table[b, j], h, :len(c)] = code_bytes(c, cache.code)
                    scales[table[b, j], h] = s
        got[name] = (torch.from_numpy(codes).to(device).view(TORCH_CODE[cache.code]),
                     torch.from_numpy(scales).to(device))
    lens = torch.tensor(cache.lens, dtype=torch.int32, device=device)
    return ibp.KVCache(got["k"][0], got["v"][0], got["k"][1], got["v"][1],
                       torch.from_numpy(table).to(device), lens)


def with_lens(cache: ibp.KVCache, lens: torch.Tensor) -> ibp.KVCache:
    return ibp.KVCache(cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, cache.table,
                       lens)


def read_all(cache: ibp.KVCache, n: int, begin=None, dtype=torch.float32):
    k = torch.empty((cache.batch, n, cache.n_heads, cache.head_dim), dtype=dtype, device="cuda")
    v = torch.empty_like(k)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ibp.kv_read(cache, k, v, begin=begin, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return {"k": k.float().cpu().numpy(), "v": v.float().cpu().numpy()}


def offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def cache_of(rng, lens, heads, page, dim, code, dtype="bf16"):
    c = ref.Cache(len(lens), heads, page, dim, code)
    for b, n in enumerate(lens):
        if n:
            c.append(b, as_float32(random_rows(rng, n, heads, dim, dtype)))
    return c
