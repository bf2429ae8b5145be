"""Oracle: rotary positions with several axes after a per-head RMS norm, fp64 (test infrastructure only).

Pair m of axis a turns by 2 pi frac(position[a] * freq[m] / 2^64); the product is formed in Python
integers, so it is exact at every position.
"""
from __future__ import annotations

import math

import numpy as np

from .rms_norm import rms_norm


def rope_axes(x, positions, freqs, axis_dims, half: bool, weight=None, eps: float = 1e-6):
    """x [B, L, heads, dh], positions int [B, L, axes] or [L, axes], freqs ints [pairs] -> fp64 [B, L, heads, dh]."""
    x = np.asarray(x, np.float64)
    B, L, H, dh = x.shape
    if weight is not None:
        x = rms_norm(x.reshape(-1, dh), weight, eps)[0].reshape(x.shape)
    positions = np.broadcast_to(np.asarray(positions), (B, L, len(axis_dims)))
    axis = [a for a, d in enumerate(axis_dims) for _ in range(d // 2)]
    n = len(axis)
    y = x.copy()
    for m in range(n):
        f = int(freqs[m]) % (1 << 64)
        angle = np.array([[2.0 * math.pi * (((int(p) * f) % (1 << 64)) / 2.0 ** 64) for p in row] for row in positions[..., axis[m]]])
        c, s = np.cos(angle)[..., None], np.sin(angle)[..., None]
        i, j = (m, m + n) if half else (2 * m, 2 * m + 1)
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., i] * s + x[..., j] * c
    return y
