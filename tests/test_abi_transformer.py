"""Host-side checks of the transformer-block operators that need no GPU: every argument error is found
before anything is launched, and the bindings refuse what the kernels do not take."""
import math

import pytest
import torch

import unet_latent_attention_b200 as sdk
from unet_latent_attention_b200 import build as sdbuild
from unet_latent_attention_b200 import fit_tanh_poly

P = 1 << 20  # a 16-byte-aligned dummy address; nothing is launched on these paths


@pytest.fixture(scope="module")
def L():
    sdbuild.build()
    return sdk.lib()


def _rms(L, fp8=False, **kw):
    a = dict(x=P, residual=0, weight=0, y=P + (1 << 16), scales=P + (1 << 18), residual_out=0, rows=4, cols=64, xs=64, rs=64, ys=64, ros=64,
             eps=1e-6, dtype=0, wf32=1, block=0)
    a.update(kw)
    head = [a[n] for n in (("x", "residual", "weight", "y", "scales", "residual_out") if fp8 else ("x", "residual", "weight", "y", "residual_out"))]
    tail = [a[n] for n in ("rows", "cols", "xs", "rs", "ys", "ros", "eps", "dtype", "wf32")] + ([a["block"]] if fp8 else [])
    return (L.sd_rms_norm_fp8 if fp8 else L.sd_rms_norm)(*head, *tail, None)


def test_rms_norm_argument_errors(L):
    assert _rms(L, rows=-1) == 1 and _rms(L, dtype=3) == 1 and _rms(L, wf32=2) == 1 and _rms(L, eps=-1.0) == 1
    assert _rms(L, eps=math.nan) == 1 and _rms(L, x=0) == 1 and _rms(L, xs=63) == 1
    assert _rms(L, residual_out=P + (1 << 19)) == 1  # without a residual
    assert _rms(L, rows=1 << 31) == 2 and _rms(L, cols=(1 << 30) + 1, xs=1 << 40, ys=1 << 40) == 2
    assert _rms(L, xs=1 << 60) == 2
    assert _rms(L, x=P + 1) == 3 and _rms(L, weight=P + 2) == 3
    assert _rms(L, y=P + 2) == 1  # partial overlap
    assert _rms(L, y=P, ys=128) == 1  # the same pointer with another stride
    assert _rms(L, residual=P + 4096, residual_out=P + (1 << 16)) == 1  # y and residual_out
    assert _rms(L, weight=P + (1 << 16)) == 1  # y over the weight
    assert _rms(L, x=0, y=0, rows=0) == 0 and _rms(L, x=0, y=0, cols=0) == 0
    assert _rms(L, fp8=True, block=16) == 2 and _rms(L, fp8=True, block=-1) == 2
    assert _rms(L, fp8=True, scales=0) == 1 and _rms(L, fp8=True, scales=P + (1 << 18) + 2) == 3
    assert _rms(L, fp8=True, y=P) == 1 and _rms(L, fp8=True, scales=P + (1 << 16)) == 1
    assert _rms(L, fp8=True, x=0, y=0, scales=0, rows=0) == 0


ROPE = ("q k q_out k_out q_weight k_weight positions freqs B L heads kv_heads dh".split()
        + [f"{t}{i}" for t in ("qs", "ks", "qos", "kos") for i in range(3)] + ["pbs"] + [f"ad{i}" for i in range(4)] + ["axes", "pairs", "dtype", "eps"])


def _rope(lib, /, **kw):
    a = dict.fromkeys(ROPE, 0)
    a.update(q=P, k=P + (1 << 16), q_out=P + (1 << 17), k_out=P + (1 << 18), positions=P + (1 << 19), freqs=P + (3 << 18), B=1, L=4, heads=2, kv_heads=1,
             dh=64, ad0=32, ad1=32, axes=2, eps=1e-6, pbs=8)
    for t, h in (("qs", 2), ("ks", 1), ("qos", 2), ("kos", 1)):
        a.update({f"{t}0": 4 * h * 64, f"{t}1": h * 64, f"{t}2": 64})
    a.update(kw)
    return lib.sd_rope_axes(sdk._ROPE_ARGS.pack(*(a[n] for n in ROPE)), None)


def test_rope_argument_errors(L):
    assert L.sd_rope_axes(None, None) == 1
    assert _rope(L, B=-1) == 1 and _rope(L, dtype=3) == 1 and _rope(L, pairs=2) == 1 and _rope(L, eps=math.inf) == 1
    assert _rope(L, dh=60) == 2 and _rope(L, dh=264) == 2 and _rope(L, axes=0) == 2 and _rope(L, axes=5) == 2
    assert _rope(L, ad0=31) == 1 and _rope(L, ad0=64) == 1 and _rope(L, ad0=30) == 2  # odd; more than dh; not a multiple of 8
    assert _rope(L, q=0) == 1 and _rope(L, k_out=0) == 1 and _rope(L, positions=0) == 1 and _rope(L, freqs=0) == 1
    assert _rope(L, q=P + 2) == 3 and _rope(L, qs1=129) == 3 and _rope(L, q_weight=P + 4) == 3 and _rope(L, freqs=P + 4) == 3
    assert _rope(L, pbs=4) == 1 and _rope(L, qs1=-128) == 2
    assert _rope(L, q_out=P + 128) == 1 and _rope(L, k_out=P + (1 << 17)) == 1 and _rope(L, q_out=P, qos1=256) == 1
    assert _rope(L, qos2=0) == 1  # the heads of an output on top of one another
    assert _rope(L, B=1 << 20, L=1 << 20) == 2
    assert _rope(L, B=0, q=0, k=0) == 0 and _rope(L, heads=0, kv_heads=0, q=0, k=0) == 0


ATT = ("q k v o bias kv_lens q_starts prefix_lens q_offsets k_offsets B heads kv_heads Lq Lk dh".split()
       + [f"{t}{i}" for t in ("qs", "ks", "vs", "os") for i in range(3)] + ["radius", "docs", "causal", "dtype", "scale", "cap"])


def _att(lib, /, **kw):
    a = dict.fromkeys(ATT, 0)
    a.update(q=P, k=P + (1 << 16), v=P + (1 << 17), o=P + (1 << 18), B=1, heads=4, kv_heads=2, Lq=8, Lk=16, dh=64, scale=0.125, cap=0.0)
    for t, h, n in (("qs", 4, 8), ("ks", 2, 16), ("vs", 2, 16), ("os", 4, 8)):
        a.update({f"{t}0": n * h * 64, f"{t}1": h * 64, f"{t}2": 64})
    a.update(kw)
    return lib.sd_attention_masked(sdk._ATTENTION_MASKED_ARGS.pack(*(a[n] for n in ATT)), None)


def test_attention_masked_argument_errors(L):
    assert L.sd_attention_masked(None, None) == 1
    assert _att(L, Lq=-1) == 1 and _att(L, dtype=2) == 1 and _att(L, causal=2) == 1 and _att(L, kv_heads=3) == 1 and _att(L, kv_heads=0) == 1
    assert _att(L, dh=60) == 2 and _att(L, dh=168) == 2 and _att(L, dh=0) == 2
    assert _att(L, scale=math.nan) == 1 and _att(L, scale=-1.0) == 2 and _att(L, cap=-1.0) == 1 and _att(L, cap=math.inf) == 1 and _att(L, cap=1e-9) == 2
    assert _att(L, bias=P, radius=1 << 29) == 1 and _att(L, bias=P, radius=-1) == 1 and _att(L, bias=P + 2) == 3
    assert _att(L, prefix_lens=P) == 1  # without causal
    assert _att(L, q_offsets=P) == 1 and _att(L, q_offsets=P, k_offsets=P, docs=0) == 1
    assert _att(L, q_offsets=P, k_offsets=P, docs=1, B=2) == 1 and _att(L, q_offsets=P, k_offsets=P, docs=1, kv_lens=P) == 1
    assert _att(L, q=0) == 1 and _att(L, v=0) == 1 and _att(L, q=P + 8) == 3 and _att(L, ks1=132) == 3 and _att(L, ks1=32) == 2
    assert _att(L, kv_lens=P + 2) == 3
    assert _att(L, o=P + 256) == 1 and _att(L, o=P + (1 << 17)) == 1 and _att(L, os2=64, os1=64) == 1
    assert _att(L, Lk=1 << 30) == 2 and _att(L, heads=1 << 17, kv_heads=1) == 2
    assert _att(L, B=0, q=0) == 0 and _att(L, Lq=0, q=0) == 0 and _att(L, heads=0, kv_heads=0, q=0) == 0


def test_bindings_refuse_on_the_host():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        sdk.sd_rms_norm(x)
    with pytest.raises(ValueError, match="bf16, fp16 or fp32"):
        sdk.sd_rms_norm(x.double())
    with pytest.raises(ValueError, match="residual"):
        sdk.sd_rms_norm(x, residual=x[:2])
    with pytest.raises(ValueError, match="residual_out needs"):
        sdk.sd_rms_norm(x, residual_out=x)
    with pytest.raises(ValueError, match="weight"):
        sdk.sd_rms_norm(x, torch.zeros(63))
    with pytest.raises(ValueError, match="block"):
        sdk.sd_rms_norm_fp8(x, block=48)
    with pytest.raises(ValueError, match="scales"):
        sdk.sd_rms_norm_fp8(x, block=32, scales=torch.zeros(4, 1))
    q, pos, f = torch.zeros(1, 4, 2, 64), torch.zeros(4, 1, dtype=torch.int32), torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        sdk.sd_rope_axes(q, None, pos, f, (64,))
    with pytest.raises(ValueError, match="positions"):
        sdk.sd_rope_axes(q, None, pos.long(), f, (64,))
    with pytest.raises(ValueError, match="freqs"):
        sdk.sd_rope_axes(q, None, pos, f[:16], (64,))
    with pytest.raises(ValueError, match="pairs"):
        sdk.sd_rope_axes(q, None, pos, f, (64,), pairs="other")
    with pytest.raises(ValueError, match="k must match"):
        sdk.sd_rope_axes(q, q[:, :2], pos, f, (64,))
    b = q.to(torch.bfloat16)
    with pytest.raises(ValueError, match="all bf16 or all fp16"):
        sdk.sd_attention_masked(q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        sdk.sd_attention_masked(b, b, b)
    with pytest.raises(ValueError, match="prefix_lens needs causal"):
        sdk.sd_attention_masked(b, b, b, prefix_lens=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="kv_lens"):
        sdk.sd_attention_masked(b, b, b, kv_lens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="go together"):
        sdk.sd_attention_masked(b, b, b, q_offsets=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="bias"):
        sdk.sd_attention_masked(b, b, b, bias=torch.zeros(4, 8))


def test_rope_frequencies():
    # pair m of an axis of d columns: theta^(-2 m / d) radians a position; the first turns one radian
    f = sdk.rope_frequencies((4, 8), theta=100.0, device="cpu")
    want = [100.0 ** (-2 * m / d) / (2 * math.pi) for d in (4, 8) for m in range(d // 2)]
    assert f.dtype == torch.int64 and all(abs(x / 2.0 ** 64 - w) < 1e-16 for x, w in zip(f.tolist(), want))
    g = sdk.rope_frequencies((4, 8), theta=100.0, inverse=True, device="cpu")
    assert all((a + b) % (1 << 64) in (0, 1, (1 << 64) - 1) or abs(a + b) < 4096 for a, b in zip(f.tolist(), g.tolist()))
    h = sdk.rope_frequencies((4, 8), theta=100.0, scale=(1.0, 0.5), device="cpu")
    assert h[:2].tolist() == f[:2].tolist() and all(abs(2 * a - b) <= 4096 for a, b in zip(h[2:].tolist(), f[2:].tolist()))
    with pytest.raises(ValueError):
        sdk.rope_frequencies((3,), device="cpu")
    with pytest.raises(ValueError):
        sdk.rope_frequencies((4, 4), scale=(1.0,), device="cpu")


def test_the_cap_polynomial_is_the_fitted_one():
    import os
    import re
    src = open(os.path.join(sdbuild.CSRC, "attention_masked.cuh")).read()
    used = [float(x) for x in re.findall(r"c\d = \{([0-9.e+-]+)f \* a\d,", src)]
    c, err = fit_tanh_poly.remez_odd()
    # the source holds them rounded to fp32: off by half a step, 2^-24 of the value, at most
    assert len(used) == len(c) == 4 and all(abs(a - b) <= 2.0 ** -24 * abs(b) for a, b in zip(used, c))
    assert err < 1.5e-7 and fit_tanh_poly.error_f32(c) < 2e-7


def test_rope_views_that_share_an_element_are_refused(L):
    # q [2, 2, 4, 64] (batch, heads, tokens, columns) in a buffer of five heads a batch, bf16, in place; k anywhere in it
    def views(k_out):
        h, b = 4 * 64, 5 * 4 * 64
        a = {}
        for t in ("qs", "ks", "qos", "kos"):
            a.update({f"{t}0": b, f"{t}1": 64, f"{t}2": h})
        return _rope(L, B=2, q=P, q_out=P, k=P + (1 << 16), k_out=k_out, **a)
    heads = [P + 2 * 4 * 64 * h for h in range(-5, 5)]
    for h in (-5, -4, 0, 1):  # a head of q, of this batch or the next
        assert views(heads[h + 5]) == 1
    for shift in (16, 2 * 64, -16):  # between two heads
        assert views(heads[5] + shift) == 1 and views(heads[6] + shift) == 1
    assert views(heads[7] - 16) == 1 and views(heads[4] + 16) == 1
