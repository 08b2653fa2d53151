"""Plain 64-bit implementations of the 8-bit paged key/value cache operators (numpy, no
code of the package): the quantisation rule, append, read, attention, eviction.

Codes follow the rule in IEEE single precision as the interface states it, so they are
compared exactly; sums (attention, its weights) are taken in 64 bits."""
from __future__ import annotations

import numpy as np

QMAX = {"int8": np.float32(127), "e4m3": np.float32(448)}


def e4m3_round(y: np.ndarray) -> np.ndarray:
    """float32 values in [-448, 448] to the nearest e4m3 value, ties to even."""
    y = np.asarray(y, np.float64)
    _, e = np.frexp(y)
    unit = np.ldexp(1.0, np.maximum(e, -5) - 4)
    return np.round(y / unit) * unit


def e4m3_values() -> np.ndarray:
    """Value of each of the 256 e4m3 bytes."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def decode(codes: np.ndarray, code: str) -> np.ndarray:
    """Bytes (uint8) to the numbers they stand for, before the scale."""
    if code == "int8":
        return codes.view(np.int8).astype(np.float64)
    return e4m3_values()[codes]


def scale_of(largest, code: str) -> np.float32:
    largest = np.float32(largest)
    if not largest > 0:
        return np.float32(0)
    s = largest * (np.float32(1) / QMAX[code])
    return np.float32(min(max(s, np.float32(2.0 ** -100)), np.float32(2.0 ** 120)))


def encode(y: np.ndarray, code: str) -> np.ndarray:
    """float32 values already times the inverse scale to coded numbers."""
    q = QMAX[code]
    with np.errstate(invalid="ignore"):
        y = np.where(np.isnan(y), np.float32(0), np.clip(y, -q, q)).astype(np.float32)
    return np.rint(y).astype(np.float64) if code == "int8" else e4m3_round(y)


class Cache:
    """values[kv][b][h]: list of pages, each (scale float32, coded numbers [tokens, D])."""

    def __init__(self, batch, heads, page, dim, code):
        self.batch, self.heads, self.page, self.dim, self.code = batch, heads, page, dim, code
        self.lens = [0] * batch
        self.tiles = {n: [[[] for _ in range(heads)] for _ in range(batch)] for n in "kv"}

    def append(self, b, rows):
        """rows: {"k": float32 [n, heads, dim], "v": ...}"""
        n = rows["k"].shape[0]
        for name in "kv":
            for h in range(self.heads):
                tiles, x, at = self.tiles[name][b][h], rows[name][:, h].astype(np.float32), 0
                while at < n:
                    off = (self.lens[b] + at) % self.page
                    m = min(n - at, self.page - off)
                    y = x[at:at + m]
                    fine = np.abs(y[np.isfinite(y)])
                    new = scale_of(fine.max() if fine.size else 0, self.code)
                    before = tiles[-1][0] if off else np.float32(0)
                    s = max(before, new)
                    inv = np.float32(1) / s if s > 0 else np.float32(0)
                    with np.errstate(invalid="ignore", over="ignore"):
                        c = encode(y * inv, self.code)
                    if off:
                        old = tiles[-1][1]
                        if s > before:
                            old = encode(old.astype(np.float32) * (before / s), self.code)
                        tiles[-1] = (s, np.concatenate([old, c]))
                    else:
                        tiles.append((s, c))
                    at += m
        self.lens[b] += n

    def values(self, name, b, h, n=None):
        """float32 values of the first n tokens."""
        t = self.tiles[name][b][h]
        if not t:
            return np.zeros((0, self.dim), np.float32)
        return np.concatenate([c.astype(np.float32) * s for s, c in t])[:n]

    def evict(self, weights, budget, recent):
        """(new cache, kept [b][h] positions): weights[b][h] arrays."""
        new = Cache(self.batch, self.heads, self.page, self.dim, self.code)
        kept = []
        for b in range(self.batch):
            row, n = [], self.lens[b]
            for h in range(self.heads):
                if n <= budget:
                    keep = np.arange(n)
                else:
                    w = np.where(np.isnan(weights[b][h][:n - recent]), -np.inf,
                                 weights[b][h][:n - recent])
                    lowest = np.isnan(weights[b][h][:n - recent])
                    order = np.lexsort((np.arange(n - recent), lowest, -w))[:budget - recent]
                    keep = np.concatenate([np.sort(order), np.arange(n - recent, n)])
                row.append(keep)
                one = Cache(1, 1, self.page, self.dim, self.code)
                one.append(0, {m: self.values(m, b, h)[keep][:, None] for m in "kv"})
                for m in "kv":
                    new.tiles[m][b][h] = one.tiles[m][0][0]
            new.lens[b] = min(n, budget)
            kept.append(row)
        return new, kept


def attention(q, keys, values, scale):
    """One sequence and K/V head in 64 bits: q [n, group, D], keys and values [t, D];
    returns out [n, group, D], lse [n, group], weights [t]."""
    n, group, dim = q.shape
    t = keys.shape[0]
    out, lse = np.zeros((n, group, dim)), np.full((n, group), -np.inf)
    weights = np.zeros(t)
    for i in range(n):
        seen = t - n + i + 1
        if seen <= 0:
            continue
        x = scale * (q[i].astype(np.float64) @ keys[:seen].astype(np.float64).T)
        top = x.max(1, keepdims=True)
        e = np.exp(x - top)
        z = e.sum(1, keepdims=True)
        p = e / z
        out[i] = p @ values[:seen].astype(np.float64)
        lse[i] = (top + np.log(z))[:, 0]
        weights[:seen] += p.sum(0)
    return out, lse, weights
