"""Oracle: RMS norm of rows with the residual's addition, and its e4m3 form, fp64 (test infrastructure only).

    h = x + residual;  y = h / sqrt(mean(h^2) + eps) * w   (Zhang and Sennrich, "Root Mean Square Layer
    Normalization");  scale of a block = max(max|y| / 448, 2^-126), q = y / scale before its rounding.
"""
from __future__ import annotations

import numpy as np


def rms_norm(x, weight, eps, residual=None):
    """(y, h) in fp64 for x [rows, C] and weight [C] or None."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    y = h / np.sqrt((h * h).mean(axis=-1, keepdims=True) + eps)
    return (y if weight is None else y * np.asarray(weight, np.float64)), h


def block_scales(y, block: int):
    """Scales [rows, ceil(C / block)] of y [rows, C] (block 0: the whole row)."""
    C = y.shape[1]
    edges = range(0, C, block or C)
    return np.stack([np.maximum(np.abs(y[:, e:e + (block or C)]).max(axis=1) / 448.0, 2.0 ** -126) for e in edges], axis=1)


def spread_scales(scales, C: int, block: int):
    """The scale of every column: [rows, C]."""
    return scales[:, np.arange(C) // (block or C)]
