"""GPU parity of sd_rms_norm and sd_rms_norm_fp8 against the fp64 oracle.

Tolerances, from the arithmetic. The sum of squares is a chain of at most 140 additions per thread and
at most 10 levels of exchange, each off by 2^-24 at most; half of that reaches the root, and the root,
the quotient and the two products add four roundings: below 100 * 2^-24 = 6e-6 relative (ARITH). An
output of type t is then off by half a step of t. An e4m3 value is off by half its step (2^-4 relative,
2^-10 below its smallest normal), at a quotient that ARITH moves twice (its scale and itself)."""
import numpy as np
import pytest
import torch

import oracle
import unet_latent_attention_b200 as sdk

pytestmark = pytest.mark.gpu

ARITH = 100 * 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _half_step(t):
    return torch.finfo(t).eps / 2


def _floor(t):  # half a step among the subnormals
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def _close(got, ref, t):
    err = np.abs(_f64(got) - ref)
    tol = np.abs(ref) * (_half_step(t) + ARITH) + _floor(t)
    assert (err <= tol).all(), float((err - tol).max())


def _fp8_close(q, scales, ref, block):
    rows, C = ref.shape
    want = oracle.block_scales(ref, block)
    s = _f64(scales).reshape(rows, -1)
    assert s.shape == want.shape and (np.abs(s - want) <= 2 * ARITH * want).all()
    v = ref / oracle.spread_scales(want, C, block)
    err = np.abs(_f64(q.float()).reshape(rows, C) - v)
    assert (err <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + 3 * ARITH * np.abs(v)).all()


def _inputs(rows, C, t, seed, dev):
    g = torch.Generator().manual_seed(seed)
    x, r = torch.randn(rows, C, generator=g), 4 * torch.randn(rows, C, generator=g)
    w = 1 + 0.1 * torch.randn(C, generator=g)
    return x.to(t).to(dev), r.to(t).to(dev), w.to(dev)


# one row and many (a CTA or a warp each), widths of every pack count, odd and long ones (read again)
SHAPES = [(1, 1), (1, 8), (3, 7), (2, 40), (5, 320), (2, 1280), (1300, 1280), (1200, 2048), (1190, 72), (1201, 333),
          (7, 2049), (3, 5000), (2, 16384), (2, 32768), (1, 70001), (1, 65544)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,C", SHAPES)
def test_plain_and_residual(cuda, rows, C, dtype):
    t = TYPES[dtype]
    x, r, w = _inputs(rows, C, t, 100 + rows + C, cuda)
    y = sdk.sd_rms_norm(x, w.to(t))
    _close(y, oracle.rms_norm(_f64(x), _f64(w.to(t)), 1e-6)[0], t)
    y, h = sdk.sd_rms_norm(x, w, 1e-5, residual=r)
    ref, hr = oracle.rms_norm(_f64(x), _f64(w), 1e-5, _f64(r))
    _close(y, ref, t)
    _close(h, hr, t)
    assert y.dtype == t and h.dtype == t


@pytest.mark.parametrize("block", [0, 32, 64, 128])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,C", [(1, 1), (2, 40), (3, 333), (2, 1280), (1300, 1280), (1201, 200), (1, 5001), (2, 16384), (1, 70001)])
def test_fp8(cuda, rows, C, dtype, block):
    t = TYPES[dtype]
    x, r, w = _inputs(rows, C, t, 500 + rows + C + block, cuda)
    q, s = sdk.sd_rms_norm_fp8(x, w, block=block)
    _fp8_close(q, s, oracle.rms_norm(_f64(x), _f64(w), 1e-6)[0], block)
    q, s, h = sdk.sd_rms_norm_fp8(x, w.to(t), residual=r, block=block)
    ref, hr = oracle.rms_norm(_f64(x), _f64(w.to(t)), 1e-6, _f64(r))
    _fp8_close(q, s, ref, block)
    _close(h, hr, t)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_in_place_and_strided_rows(cuda, dtype):
    t = TYPES[dtype]
    x, r, w = _inputs(1300, 1280, t, 7, cuda)
    ref, hr = oracle.rms_norm(_f64(x), _f64(w), 1e-6, _f64(r))
    y, h = sdk.sd_rms_norm(x, w, residual=r, out=x, residual_out=r)
    assert y is x and h is r
    _close(x, ref, t)
    _close(r, hr, t)
    # columns of a wider buffer, at odd offsets (no 16-byte alignment) and even ones; the rest stays
    for off in (8, 3):
        big = torch.randn(2, 50, 512, generator=torch.Generator().manual_seed(9)).to(t).to(cuda)
        out = torch.full_like(big, 5.0)
        xs, ys = big[..., off:off + 200], out[..., off:off + 200]
        sdk.sd_rms_norm(xs, out=ys)
        _close(ys.reshape(-1, 200), oracle.rms_norm(_f64(xs).reshape(-1, 200), None, 1e-6)[0], t)
        assert (out[..., :off] == 5).all() and (out[..., off + 200:] == 5).all()
    # two column slices of one buffer: in from one, out to the other
    buf = torch.randn(40, 128, generator=torch.Generator().manual_seed(10)).to(t).to(cuda)
    ref = oracle.rms_norm(_f64(buf[:, :64]), None, 1e-6)[0]
    sdk.sd_rms_norm(buf[:, :64], out=buf[:, 64:])
    _close(buf[:, 64:], ref, t)


def test_zero_rows_nan_and_infinity(cuda):
    x = torch.randn(6, 256, generator=torch.Generator().manual_seed(3)).to(cuda)
    x[1] = 0
    x[2, 130] = float("nan")
    x[3, 5] = float("inf")
    x[4] = torch.finfo(torch.float32).tiny / 4
    y = sdk.sd_rms_norm(x)
    assert (y[1] == 0).all() and y[2].isnan().all() and y[3, 5].isnan() and (y[3, 6:] == 0).all()
    for block in (0, 128):
        q, s = sdk.sd_rms_norm_fp8(x, block=block)
        assert (q[1].float() == 0).all() and (s[1] == 2.0 ** -126).all()
        assert s[2].isnan().all() and q[2].float().isnan().all()
        assert s[3, 0].isnan() and q[3, :128].float().isnan().all()
        assert q[0].float().isfinite().all() and q[4].float().isfinite().all() and s[5].isfinite().all()
    assert torch.equal(sdk.sd_rms_norm(x[:1]), y[:1])


def test_empty(cuda):
    assert sdk.sd_rms_norm(torch.zeros(0, 64, device=cuda)).shape == (0, 64)
    q, s = sdk.sd_rms_norm_fp8(torch.zeros(0, 64, device=cuda), block=32)
    assert q.shape == (0, 64) and s.shape == (0, 2)


def test_overlaps_are_refused(cuda):
    x = torch.zeros(4, 128, device=cuda)
    for kw in (dict(out=x.view(-1)[64:-64].view(3, 128)),):
        with pytest.raises((sdk.SDError, ValueError)):
            sdk.sd_rms_norm(x[:3], **kw)
    big = torch.zeros(8, 128, device=cuda)
    with pytest.raises(sdk.SDError, match="overlaps"):
        sdk.sd_rms_norm(big[0:4], out=big[1:5])
    with pytest.raises(sdk.SDError, match="overlaps"):
        sdk.sd_rms_norm(big[0:4], residual=big[4:8], residual_out=big[3:7])
    with pytest.raises(sdk.SDError, match="overlaps"):
        sdk.sd_rms_norm_fp8(x, out=x.view(torch.float8_e4m3fn)[:, :128])


def test_captured_and_on_another_stream(cuda):
    x, r, w = _inputs(300, 640, torch.bfloat16, 11, cuda)
    want = sdk.sd_rms_norm_fp8(x, w, residual=r, block=64)
    out = [torch.empty_like(t) for t in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            sdk.sd_rms_norm_fp8(x, w, residual=r, block=64, out=out[0], scales=out[1], residual_out=out[2])
        g.replay()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(out, want):
        assert torch.equal(a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a,
                           b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("C", [1 << 24, (1 << 22) + 7])
def test_wide_rows_of_equal_values(cuda, C, dtype):
    # equal terms round the same way at every addition: a long chain of them drifts
    t = TYPES[dtype]
    for value in (1.1, 3.3):
        x = torch.full((1, C), value, dtype=t, device=cuda)
        v = float(x[0, 0])
        want = v / np.sqrt(v * v + 1e-6)
        y = sdk.sd_rms_norm(x)
        assert ((y.double() - want).abs() <= want * (_half_step(t) + ARITH)).all()
        q, s = sdk.sd_rms_norm_fp8(x, block=0)
        assert (q.float() == 448).all() and abs(float(s) - want / 448) <= 2 * ARITH * want / 448
        x[0, ::2] *= 2
        a, b = float(x[0, 0]), v
        n = (C + 1) // 2
        rms = np.sqrt((n * a * a + (C - n) * b * b) / C + 1e-6)
        y, h = sdk.sd_rms_norm(x, residual=torch.zeros_like(x))
        assert ((y[0, ::2].double() - a / rms).abs() <= a / rms * (_half_step(t) + ARITH)).all() and torch.equal(h, x)
        assert ((y[0, 1::2].double() - b / rms).abs() <= b / rms * (_half_step(t) + ARITH)).all()
