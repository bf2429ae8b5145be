"""Fits the polynomial that caps attention scores (run to reproduce its constants).

sd_attention_masked evaluates tanh(u), u = score / cap, as u P(u^2) on the FMA pipe while |u| <= 1/2 (and
from two special-function results beyond). P is the polynomial of degree 3 whose largest absolute error
of u P(u^2) on [0, 1/2] is smallest, found by the Remez exchange algorithm (Remez, 1934).

    python -m unet_latent_attention_b200.fit_tanh_poly
"""
from __future__ import annotations

import numpy as np


def remez_odd(deg: int = 3, hi: float = 0.5, iters: int = 60):
    """Coefficients p0..p_deg and the largest |u P(u^2) - tanh(u)| on [0, hi]."""
    n = deg + 1
    x = 0.5 * hi * (1 - np.cos(np.pi * (np.arange(n + 1) + 0.5) / (n + 1)))
    grid = np.linspace(1e-4, hi, 200001)
    for _ in range(iters):
        A = np.hstack([x[:, None] ** (2 * np.arange(n) + 1), (-1.0) ** np.arange(n + 1)[:, None]])
        c = np.linalg.solve(A, np.tanh(x))[:n]
        err = np.tanh(grid) - (grid[:, None] ** (2 * np.arange(n) + 1)) @ c
        cuts = np.concatenate([[0], np.nonzero(np.diff(np.sign(err)))[0] + 1, [len(grid)]])
        ext = [a + int(np.argmax(np.abs(err[a:b]))) for a, b in zip(cuts[:-1], cuts[1:]) if b > a]
        if len(ext) < n + 1:
            break
        while len(ext) > n + 1:
            ext = ext[1:] if abs(err[ext[0]]) < abs(err[ext[-1]]) else ext[:-1]
        x = grid[ext]
    return c, float(np.abs(err).max())


def error_f32(c, hi: float = 0.5):
    """The largest error with fp32 coefficients and fp32 evaluation (one rounding per multiply-add)."""
    c = np.asarray(c, np.float32)
    u = np.linspace(-hi, hi, 1000001).astype(np.float32)
    z = u * u
    p = np.full_like(u, c[-1])
    for k in range(len(c) - 2, -1, -1):
        p = (p.astype(np.float64) * z + c[k]).astype(np.float32)
    return float(np.abs((p * u).astype(np.float64) - np.tanh(u.astype(np.float64))).max())


if __name__ == "__main__":
    c, e = remez_odd()
    print("p0..p3 =", ", ".join(f"{float(np.float32(v)):.9e}f" for v in c))
    print(f"max absolute error: {e:.3e} (real arithmetic), {error_f32(c):.3e} (fp32)")
