"""Frequency tables of sd_rope_axes.

Pair m of an axis of d columns turns by theta^(-2 m / d) radians per position (Su et al., "RoFormer:
Enhanced Transformer with Rotary Position Embedding"). The kernel takes the frequency as a 64-bit
fraction of a turn, so that positions of any size keep their angle.
"""
from __future__ import annotations

import math

ONE_TURN = 1 << 64


def turns_to_fixed(turns):
    """Turns per position (floats) -> the two's complement of their 64-bit fractions, as Python ints in
    [-2^63, 2^63)."""
    out = []
    for t in turns:
        f = round((t - math.floor(t)) * ONE_TURN) % ONE_TURN
        out.append(f - ONE_TURN if f >= ONE_TURN // 2 else f)
    return out


def rope_frequencies(axis_dims, theta: float = 10000.0, scale=1.0, inverse: bool = False, device="cuda"):
    """int64 tensor [sum(axis_dims) / 2] of the frequencies of all pairs, axis after axis.

    ``scale`` multiplies the positions (one number, or one per axis: 0.5 squeezes twice as many positions
    into the trained range). ``inverse`` negates the angles: the call then undoes the rotation."""
    import torch
    axis_dims = list(axis_dims)
    scales = list(scale) if hasattr(scale, "__len__") else [scale] * len(axis_dims)
    if len(scales) != len(axis_dims):
        raise ValueError("scale must be one number or one per axis")
    turns = []
    for d, s in zip(axis_dims, scales):
        if d < 0 or d % 2:
            raise ValueError("each axis takes an even number of columns")
        turns += [(-s if inverse else s) * theta ** (-2.0 * m / d) / (2.0 * math.pi) for m in range(d // 2)]
    return torch.tensor(turns_to_fixed(turns), dtype=torch.int64, device=device)
