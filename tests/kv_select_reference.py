"""Plain selection of pages (numpy, no code of the package): bounds, scores and columns as the
interface states them, and attention over the selected pages in 64 bits."""
from __future__ import annotations

import numpy as np

import kv_reference as ref


def bounds(codes: np.ndarray, code: str):
    """Least and largest of a page's coded numbers [tokens, D] as whole numbers."""
    lo, hi = codes.min(0).astype(np.float64), codes.max(0).astype(np.float64)
    if code == "e4m3":
        lo, hi = np.floor(lo * 127 / 448), np.ceil(hi * 127 / 448)
    return np.clip(lo, -127, 127).astype(np.int64), np.clip(hi, -127, 127).astype(np.int64)


def whole(row: np.ndarray):
    """A query row in whole numbers, and the exponent e."""
    row = np.where(np.isnan(row), np.float32(0), row).astype(np.float32)
    most = np.abs(row).max()
    with np.errstate(over="ignore"):
        e = 100 if np.isinf(most) else int(np.clip(np.frexp(most)[1] - 1, -100, 100))
        return np.clip(np.rint(row.astype(np.float64) * 2.0 ** (6 - e)), -127, 127).astype(np.int64), e


def scores(cache: ref.Cache, b, h, rows: np.ndarray):
    """float32 score of every page of sequence b, head h, for rows [m, D]."""
    out = []
    for s, codes in cache.tiles["k"][b][h]:
        lo, hi = bounds(codes, cache.code)
        best = -np.inf
        for row in rows:
            n, e = whole(row)
            best = max(best, float(np.maximum(n * lo, n * hi).sum()) * 2.0 ** (e - 6))
        with np.errstate(over="ignore", invalid="ignore"):
            out.append(np.float32(best) * np.float32(s))
    return np.array(out, np.float32)


def columns(cache: ref.Cache, b, h, rows: np.ndarray, n: int, pages: int):
    """Columns selected for n query positions (rows [n * group, D]), rising."""
    length, P = cache.lens[b], cache.page
    all_ = -(-length // P)
    if n == 0:
        return []
    if all_ <= pages:
        return list(range(all_))
    own = range(min(max(length - n, 0) // P, all_ - 1), all_)
    x = scores(cache, b, h, rows)
    open_ = [c for c in range(1, own[0])]
    key = lambda c: (not np.isnan(x[c]), x[c] if not np.isnan(x[c]) else 0)  # noqa: E731
    order = sorted(open_, key=lambda c: (-key(c)[0], -key(c)[1], c))[:pages - 1 - len(own)]
    return sorted([0] + order) + list(own)


def attention(cache: ref.Cache, b, h, q, cols, scale):
    """q [n, group, D] over the tokens of the pages cols; out [n, group, D], lse [n, group]."""
    n, group, dim = q.shape
    length, P = cache.lens[b], cache.page
    t = np.concatenate([np.arange(c * P, min(c * P + P, length)) for c in cols] or [np.zeros(0, int)]).astype(int)
    k, v = cache.values("k", b, h)[t], cache.values("v", b, h)[t]
    out, lse, size, least = np.zeros((n, group, dim)), np.full((n, group), -np.inf), np.zeros((n, group, dim)), 0.0
    for i in range(n):
        seen = t <= length - n + i
        if not seen.any():
            continue
        x = scale * (q[i].astype(np.float64) @ k[seen].astype(np.float64).T)
        top = x.max(1, keepdims=True)
        e = np.exp(x - top)
        z = e.sum(1, keepdims=True)
        out[i], lse[i] = (e / z) @ v[seen], (top + np.log(z))[:, 0]
        size[i] = (e / z) @ np.abs(v[seen])
        least = max(least, (abs(scale) * (np.abs(q[i].astype(np.float64)) @ np.abs(k[seen]).T.astype(np.float64))).max())
    return out, lse, size, least
