"""Plain rotation of positions (numpy, no code of the package), in the steps of single
precision that the interface states: every product and every sum rounded once."""
from __future__ import annotations

import numpy as np


def table(n_positions, dim, base=10000.0):
    angle = np.arange(n_positions, dtype=np.float64)[:, None] * \
        float(base) ** (-np.arange(dim // 2, dtype=np.float64) / (dim // 2))
    return np.stack([np.cos(angle), np.sin(angle)], 2).astype(np.float32)


def rotated(x, turns, positions, axis, interleaved):
    """x [n, heads, D] float32; turns [positions, dim/2, 2]; positions [n, axes]."""
    x, y = np.asarray(x, np.float32), np.array(x, np.float32)
    pairs = turns.shape[1]
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        at = np.clip(positions[:, axis[i]], 0, turns.shape[0] - 1)
        c, s = turns[at, i, 0][:, None], turns[at, i, 1][:, None]
        with np.errstate(invalid="ignore", over="ignore"):
            y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
            y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y
