"""Oracle: attention with masks, a tanh cap and a bias by distance, fp64 (test infrastructure only).

The definition, one query at a time over the keys that it sees; a key that is not seen is left out, so its
values cannot matter. See ``attention`` for the form without masks.
"""
from __future__ import annotations

import numpy as np

from .attention import _f64


def seen_keys(Lq, Lk, causal=False, length=None, start=None, prefix=0):
    """(bool [Lq, Lk], distance [Lq, Lk]) of one sequence: key j is seen if j < length and (not causal or
    j <= start + i or j < prefix); distance = j - (start + i)."""
    length = Lk if length is None else min(max(int(length), 0), Lk)
    start = Lk - Lq if start is None else int(start)
    i, j = np.arange(Lq)[:, None], np.arange(Lk)[None, :]
    dist = j - (i + start)
    see = (j < length) & np.ones_like(i, bool)
    return (see & ((dist <= 0) | (j < prefix)) if causal else see), dist


def _one(q, k, v, see, dist, scale, cap, bias_row):
    """o [Lq, dh] and sum_j p_j |v_j| [Lq, dh] of one head of one sequence."""
    t = scale * (q @ k.T)
    if cap:
        t = cap * np.tanh(t / cap)
    if bias_row is not None:
        R = len(bias_row) // 2
        t = t + bias_row[np.clip(dist, -R, R) + R]
    o, a = np.zeros((q.shape[0], v.shape[1])), np.zeros((q.shape[0], v.shape[1]))
    for i in range(q.shape[0]):
        js = np.nonzero(see[i])[0]
        if not len(js) or (t[i, js] == -np.inf).all():
            continue
        p = np.exp(t[i, js] - t[i, js].max())
        p /= p.sum()
        o[i], a[i] = p @ v[js], p @ np.abs(v[js])
    return o, a


def attention_masked(q, k, v, scale=None, causal=False, cap=0.0, bias=None, kv_lens=None, q_starts=None, prefix_lens=None,
                     q_offsets=None, k_offsets=None, out=None):
    """(o, sum_j p_j |v_j|), fp64 [B, heads, Lq, dh]; arguments as sd_attention_masked, heads first.
    Rows in no document keep ``out`` (zeros if it is None)."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, H, Lq, dh = q.shape
    KV, Lk = k.shape[1], k.shape[2]
    scale = 1.0 / np.sqrt(dh) if scale is None else scale
    o = np.zeros_like(q) if out is None else _f64(out).copy()
    a = np.zeros_like(q)
    bias = None if bias is None else _f64(bias)
    parts = []  # batch row, queries, keys, seen keys, distances
    if q_offsets is not None:
        for d in range(len(q_offsets) - 1):
            q0, q1, k0, k1 = (int(x) for x in (q_offsets[d], q_offsets[d + 1], k_offsets[d], k_offsets[d + 1]))
            parts.append((0, q0, q1, k0, k1, seen_keys(q1 - q0, k1 - k0, causal, None, None if q_starts is None else q_starts[d],
                                                       0 if prefix_lens is None else int(prefix_lens[d]))))
    else:
        for b in range(B):
            parts.append((b, 0, Lq, 0, Lk, seen_keys(Lq, Lk, causal, None if kv_lens is None else kv_lens[b],
                                                     None if q_starts is None else q_starts[b],
                                                     0 if prefix_lens is None else int(prefix_lens[b]))))
    with np.errstate(invalid="ignore"):
        for b, q0, q1, k0, k1, (see, dist) in parts:
            for h in range(H):
                g = h // (H // KV)
                o[b, h, q0:q1], a[b, h, q0:q1] = _one(q[b, h, q0:q1], k[b, g, k0:k1], v[b, g, k0:k1], see, dist, scale, cap,
                                                      None if bias is None else bias[h])
    return o, a
