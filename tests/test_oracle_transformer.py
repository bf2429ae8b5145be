"""Pins of the transformer-block oracles: closed forms, invariants and independent routines (CPU)."""
import math

import numpy as np
import pytest

import oracle
import synth_inputs as si


def test_rms_norm_closed_forms():
    y, h = oracle.rms_norm([[3.0, 4.0]], [2.0, 0.5], 0.0, [[0.0, 0.0]])
    r = math.sqrt(12.5)
    assert np.allclose(y, [[6 / r, 2 / r]], rtol=1e-15) and np.array_equal(h, [[3.0, 4.0]])
    x = si.normal((5, 37), 1).astype(np.float64)
    y, _ = oracle.rms_norm(x, None, 0.0)
    assert np.allclose((y ** 2).mean(axis=1), 1.0, rtol=1e-14)
    assert np.allclose(oracle.rms_norm(7 * x, None, 0.0)[0], y, rtol=1e-14)  # scale does not matter without eps
    assert np.allclose(oracle.rms_norm(x, None, 1e-3, -x)[0], 0.0)


def test_block_scales():
    y = np.array([[448.0, -896.0, 1.0, 0.0, 0.0]])
    assert np.allclose(oracle.block_scales(y, 0), [[2.0]])
    s = oracle.block_scales(np.pad(y, ((0, 0), (0, 60))), 32)
    assert s.shape == (1, 3) and s[0, 0] == 2.0 and s[0, 1] == s[0, 2] == 2.0 ** -126
    assert oracle.spread_scales(s, 65, 32).shape == (1, 65) and oracle.spread_scales(s, 65, 32)[0, 31] == 2.0


@pytest.mark.parametrize("half", [False, True])
def test_rope_quarter_turns_and_relative_positions(half):
    x = np.arange(1.0, 5.0).reshape(1, 1, 1, 4)
    quarter = [1 << 62, 1 << 62]
    y = oracle.rope_axes(x, [[[1]]], quarter, (4,), half)
    want = [-3.0, -4.0, 1.0, 2.0] if half else [-2.0, 1.0, -4.0, 3.0]
    assert np.allclose(y.ravel(), want, atol=1e-15)
    assert np.allclose(oracle.rope_axes(x, [[[2 ** 31 - 1]]], quarter, (4,), half), oracle.rope_axes(x, [[[3]]], quarter, (4,), half), atol=1e-15)
    # a query's product with a key depends on the distance only, axis by axis
    q, k = (si.normal((1, 1, 1, 16), s).astype(np.float64) for s in (2, 3))
    f = [int(t * 2 ** 64) for t in (0.15, 0.01, 0.3, 0.07, 0.001, 0.2, 0.11, 0.05)]
    dots = [(oracle.rope_axes(q, [[[a, b]]], f, (8, 8), half) * oracle.rope_axes(k, [[[a + 5, b - 3]]], f, (8, 8), half)).sum()
            for a, b in ((0, 0), (17, 40), (100000, -7))]
    assert np.allclose(dots, dots[0], rtol=1e-9)


def test_rope_norm_and_untouched_columns():
    x = si.normal((1, 2, 3, 12), 4).astype(np.float64)
    w = 1 + 0.1 * si.normal((12,), 5).astype(np.float64)
    y = oracle.rope_axes(x, [[0], [9]], [1 << 60, 1 << 59], (4,), False, w, 1e-6)
    n = oracle.rms_norm(x.reshape(-1, 12), w, 1e-6)[0].reshape(x.shape)
    assert np.allclose(y[:, 0], n[:, 0], rtol=1e-15) and np.allclose(y[..., 4:], n[..., 4:], rtol=1e-15)
    assert np.allclose((y ** 2).sum(-1), (n ** 2).sum(-1), rtol=1e-13)


def _qkv(B, H, KV, Lq, Lk, dh, seed):
    return (si.normal((B, H, Lq, dh), seed).astype(np.float64), si.normal((B, KV, Lk, dh), seed + 1).astype(np.float64),
            si.normal((B, KV, Lk, dh), seed + 2).astype(np.float64))


def test_attention_masked_without_masks_is_attention():
    q, k, v = _qkv(2, 3, 3, 5, 7, 8, 10)
    o, a = oracle.attention_masked(q, k, v)
    assert np.allclose(o, oracle.attention(q, k, v), rtol=1e-13) and (a >= np.abs(o) - 1e-15).all()
    q, k, v = _qkv(1, 4, 2, 5, 7, 8, 11)  # grouped heads
    assert np.allclose(oracle.attention_masked(q, k, v)[0], oracle.attention(q, np.repeat(k, 2, 1), np.repeat(v, 2, 1)), rtol=1e-13)


def test_attention_masked_hand_case():
    # one query at position 1 of three keys with equal scores: causal sees two, a prefix of 3 all, a length of 1 one
    q, k = np.zeros((1, 1, 1, 2)), np.zeros((1, 1, 3, 2))
    v = np.array([[1.0, 0.0], [3.0, 0.0], [8.0, 4.0]])[None, None]
    f = lambda **kw: oracle.attention_masked(q, k, v, causal=True, q_starts=[1], **kw)[0].ravel()  # noqa: E731
    assert np.allclose(f(), [2.0, 0.0]) and np.allclose(f(prefix_lens=[3]), [4.0, 4.0 / 3]) and np.allclose(f(kv_lens=[1]), [1.0, 0.0])
    assert np.allclose(f(kv_lens=[0]), [0.0, 0.0])
    # a bias of log 3 on the key one behind: weights 3 : 1
    bias = np.log(np.array([[1.0, 3.0, 1.0, 1.0, 1.0]]))
    assert np.allclose(f(bias=bias), [(3 * 1 + 3) / 4, 0.0])
    # a cap of 1 on scores of 0 and 20: exp(tanh(20)) to 1
    q1, k1 = np.full((1, 1, 1, 1), 20.0), np.array([[0.0], [1.0]])[None, None]
    w = math.exp(math.tanh(20.0))
    assert np.allclose(oracle.attention_masked(q1, k1, k1, scale=1.0, cap=1.0)[0].ravel(), [w / (1 + w)])


def test_attention_masked_documents_are_separate_calls():
    q, k, v = _qkv(1, 2, 1, 9, 11, 8, 12)
    qo, ko = [1, 4, 4, 8], [0, 3, 7, 11]
    out = np.full((1, 2, 9, 8), 5.0)
    o, _ = oracle.attention_masked(q, k, v, causal=True, q_offsets=qo, k_offsets=ko, out=out)
    for d in range(3):
        s = slice(qo[d], qo[d + 1])
        part, _ = oracle.attention_masked(q[:, :, s], k[:, :, ko[d]:ko[d + 1]], v[:, :, ko[d]:ko[d + 1]], causal=True)
        assert np.array_equal(o[:, :, s], part)
    assert (o[:, :, 0] == 5).all() and (o[:, :, 8] == 5).all()


def test_unseen_values_do_not_matter_to_the_oracle():
    q, k, v = _qkv(1, 1, 1, 4, 6, 8, 13)
    o, _ = oracle.attention_masked(q, k, v, kv_lens=[4])
    k[:, :, 4:], v[:, :, 4:] = np.nan, np.inf
    assert np.array_equal(oracle.attention_masked(q, k, v, kv_lens=[4])[0], o)
