"""GPU parity of sd_rope_axes against the fp64 oracle (angles formed in exact integers).

Tolerance: the angle is cut to 2^-32 turns and rounded to fp32 half turns (2^-25 * pi = 9.4e-8 rad), sincospi
is off by an ulp (6e-8): each of cos and sin by less than 1.6e-7. With the roundings of the product and of
the norm (a chain of 8 and 5 additions, the root, two products: 11 * 2^-24) a value of a pair (u, v) is off
by less than 1e-6 (|u| + |v|), and then by half a step of its type."""
import numpy as np
import pytest
import torch

import oracle
import unet_latent_attention_b200 as sdk

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _check(got, x, pos, freqs, axes, half, w, eps=1e-6):
    ref = oracle.rope_axes(_f64(x), pos.cpu().numpy(), freqs.tolist(), axes, half, None if w is None else _f64(w), eps)
    n = oracle.rms_norm(_f64(x).reshape(-1, x.shape[-1]), _f64(w), eps)[0].reshape(x.shape) if w is not None else _f64(x)
    t = got.dtype
    most = np.abs(n).max(axis=-1, keepdims=True)
    tol = np.abs(ref) * torch.finfo(t).eps / 2 + 2e-6 * most + torch.finfo(t).smallest_normal * torch.finfo(t).eps
    err = np.abs(_f64(got) - ref)
    assert (err <= tol).all(), float((err - tol).max())


def _inputs(B, L, H, KV, dh, t, seed, dev, axes, far=100):
    g = torch.Generator().manual_seed(seed)
    q, k = torch.randn(B, L, H, dh, generator=g).to(t).to(dev), torch.randn(B, L, KV, dh, generator=g).to(t).to(dev)
    pos = torch.randint(-far, far, (B, L, len(axes)), generator=g, dtype=torch.int32).to(dev)
    w = [(1 + 0.2 * torch.randn(dh, generator=g)).to(dev) for _ in range(2)]
    return q, k, pos, w


CASES = [(8, (8,)), (40, (8, 16, 16)), (64, (64,)), (64, (16, 24, 24)), (72, (24, 24, 24)), (80, (16, 32, 32)), (128, (44, 42, 42)),
         (128, (32, 32)), (160, (32, 64, 64)), (256, (256,)), (64, (8, 0, 16, 16)), (24, (0,))]


@pytest.mark.parametrize("pairs", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dh,axes", CASES, ids=[f"{d}-{'_'.join(map(str, a))}" for d, a in CASES])
def test_shapes(cuda, dh, axes, dtype, pairs):
    t = TYPES[dtype]
    freqs = sdk.rope_frequencies(axes)
    for (B, L, H, KV), norm in (((1, 1, 1, 1), False), ((2, 37, 5, 1), True), ((2, 9, 6, 3), False)):
        q, k, pos, (wq, wk) = _inputs(B, L, H, KV, dh, t, dh + L, cuda, axes)
        qo, ko = sdk.sd_rope_axes(q, k, pos, freqs, axes, pairs=pairs, q_weight=wq if norm else None, k_weight=wk if norm else None)
        _check(qo, q, pos, freqs, axes, pairs == "half", wq if norm else None)
        _check(ko, k, pos, freqs, axes, pairs == "half", wk if norm else None)


@pytest.mark.parametrize("pairs", ["interleaved", "half"])
def test_far_positions(cuda, pairs):
    # an angle formed in fp32 is radians off at these positions
    axes = (32, 32)
    q, k, _, _ = _inputs(1, 8, 2, 2, 64, torch.float32, 5, cuda, axes)
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31], [10 ** 9, 123456789], [1, -1], [0, 0], [65535, 10 ** 7], [-7, 2 ** 30], [2 ** 24 + 1, 99], [3, 4]],
                       dtype=torch.int32, device=cuda)
    freqs = sdk.rope_frequencies(axes)
    qo, ko = sdk.sd_rope_axes(q, k, pos, freqs, axes, pairs=pairs)
    _check(qo, q, pos[None], freqs, axes, pairs == "half", None)
    assert torch.equal(qo[:, 3], q[:, 3])  # position 0 turns nothing


def test_many_rows_take_four_heads_a_thread(cuda):
    axes = (16, 24, 24)
    q, k, pos, (wq, wk) = _inputs(1, 7000, 16, 7, 64, torch.bfloat16, 6, cuda, axes)
    freqs = sdk.rope_frequencies(axes)
    qo, ko = sdk.sd_rope_axes(q, k, pos, freqs, axes, q_weight=wq, k_weight=wk)
    rows = torch.tensor([0, 1, 3499, 6998, 6999], device=cuda)
    _check(qo[:, rows], q[:, rows], pos[:, rows], freqs, axes, False, wq)
    _check(ko[:, rows], k[:, rows], pos[:, rows], freqs, axes, False, wk)
    # the same rows in a short call (one head a thread) have the same bits
    qs, ks = sdk.sd_rope_axes(q[:, :16], k[:, :16], pos[:, :16].contiguous(), freqs, axes, q_weight=wq, k_weight=wk)
    assert torch.equal(qs, qo[:, :16]) and torch.equal(ks, ko[:, :16])


@pytest.mark.parametrize("H,KV", [(1, 1), (2, 2), (3, 1), (1, 0), (4, 3), (8, 1), (1, 6), (40, 10)])
@pytest.mark.parametrize("dh", [16, 64, 128, 160])
def test_every_head_of_many_tokens_is_written(cuda, dh, H, KV):
    # however the heads are dealt to the threads: every value, against the rotation in torch's fp64
    axes = (dh // 2, dh // 2)
    L = 12001
    q, k, pos, (wq, wk) = _inputs(1, L, H, max(KV, 1), dh, torch.float16, 60 + dh + H, cuda, axes)
    freqs = sdk.rope_frequencies(axes)
    for norm in (False, True):
        qo, ko = (torch.full_like(x, float("nan")) for x in (q, k))
        sdk.sd_rope_axes(q, k if KV else None, pos, freqs, axes, q_weight=wq if norm else None, k_weight=wk if norm else None,
                         q_out=qo, k_out=ko if KV else None)
        for x, y, w in ((q, qo, wq), (k, ko, wk))[:2 if KV else 1]:
            axis = torch.tensor([a for a, d in enumerate(axes) for _ in range(d // 2)], device=cuda)
            angle = 2 * np.pi * (pos.double()[..., axis] * (freqs.double() * 2.0 ** -64))[:, :, None]
            n = x.double()
            if norm:
                n = n / (n.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
            a, b = n[..., 0::2], n[..., 1::2]
            ref = torch.stack((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1).flatten(-2)
            tol = ref.abs() * 2.0 ** -11 + 2e-6 * n.abs().amax(-1, keepdim=True) + 2.0 ** -24
            assert ((y.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_fused_projection_in_place_and_layouts(cuda, dtype):
    t, axes, half = TYPES[dtype], (16, 24, 24), True
    B, L, H, KV, dh = 2, 33, 4, 2, 64
    g = torch.Generator().manual_seed(8)
    rows = torch.randn(B, L, H + 2 * KV, dh, generator=g).to(t).to(cuda)
    before = rows.clone()
    pos = torch.randint(0, 64, (L, 3), generator=g, dtype=torch.int32).to(cuda)  # shared by the batch
    freqs = sdk.rope_frequencies(axes, theta=1000.0, scale=(1.0, 0.5, 0.5))
    w = (1 + 0.2 * torch.randn(dh, generator=g)).to(cuda)
    q, k = rows[:, :, :H], rows[:, :, H:H + KV]
    qo, ko = sdk.sd_rope_axes(q, k, pos, freqs, axes, pairs="half", q_weight=w)
    _check(qo, q, pos[None], freqs, axes, half, w)
    _check(ko, k, pos[None], freqs, axes, half, None)
    # heads-first views, one tensor only
    q2, none = sdk.sd_rope_axes(q.transpose(1, 2), None, pos, freqs, axes, pairs="half", layout="bhld", q_weight=w)
    assert none is None and torch.equal(q2.transpose(1, 2), qo)
    # in place on the projection's rows: the values stay
    sdk.sd_rope_axes(q, k, pos, freqs, axes, pairs="half", q_weight=w, q_out=q, k_out=k)
    assert torch.equal(rows[:, :, :H], qo) and torch.equal(rows[:, :, H:H + KV], ko)
    assert torch.equal(rows[:, :, H + KV:], before[:, :, H + KV:])
    # both outputs in the rows of one buffer
    out = torch.zeros(B, L, H + KV, dh, dtype=t, device=cuda)
    sdk.sd_rope_axes(before[:, :, :H], before[:, :, H:H + KV], pos, freqs, axes, pairs="half", q_weight=w, q_out=out[:, :, :H], k_out=out[:, :, H:])
    assert torch.equal(out[:, :, :H], qo) and torch.equal(out[:, :, H:], ko)


def test_keys_alone_and_token_slices_of_fused_rows(cuda):
    # heads = 0 (a call of the C interface): k alone, few tokens and many
    axes, dh = (64,), 64
    freqs = sdk.rope_frequencies(axes)
    for L in (1, 9, 9000):
        _, k, pos, _ = _inputs(1, L, 1, 3, dh, torch.bfloat16, 20 + L, cuda, axes)
        want, _ = sdk.sd_rope_axes(k, None, pos, freqs, axes)
        out = torch.zeros_like(k)
        s = (L * 3 * dh, 3 * dh, dh)
        args = sdk._ROPE_ARGS.pack(0, k.data_ptr(), 0, out.data_ptr(), 0, 0, pos.data_ptr(), freqs.data_ptr(), 1, L, 0, 3, dh, 0, 0, 0, *s, 0, 0, 0, *s,
                                   L, 64, 0, 0, 0, 1, 0, 0, 1e-6)
        assert sdk.lib().sd_rope_axes(args, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(out, want)
    # the later tokens of a fused projection's rows, in place: q and k interleave but do not meet
    rows = torch.randn(3, 20, 7, dh, generator=torch.Generator().manual_seed(21)).to(torch.bfloat16).to(cuda)
    q, k = rows[:, 5:, :4], rows[:, 5:, 4:6]
    pos = torch.arange(15, dtype=torch.int32, device=cuda).view(15, 1)
    before = rows.clone()
    qo, ko = sdk.sd_rope_axes(q, k, pos, freqs, axes)
    sdk.sd_rope_axes(q, k, pos, freqs, axes, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(rows[:, :5], before[:, :5]) and torch.equal(rows[:, :, 6:], before[:, :, 6:])
    with pytest.raises(sdk.SDError, match="overlaps"):
        sdk.sd_rope_axes(rows[:, 5:, :4], rows[:, 5:, 3:5], pos, freqs, axes, q_out=rows[:, 5:, :4], k_out=rows[:, 5:, 3:5])


def test_inverse_and_gradient(cuda):
    # the inverse table undoes the rotation, and the rotation's gradient is the inverse applied to it
    axes = (16, 24, 24)
    q, _, pos, _ = _inputs(1, 19, 3, 1, 64, torch.float32, 12, cuda, axes)
    f, inv = sdk.rope_frequencies(axes), sdk.rope_frequencies(axes, inverse=True)
    y, _ = sdk.sd_rope_axes(q, None, pos, f, axes)
    back, _ = sdk.sd_rope_axes(y, None, pos, inv, axes)
    assert (back - q).abs().max() <= 4e-6 * q.abs().max()
    g = torch.randn(y.shape, generator=torch.Generator().manual_seed(13)).to(cuda)
    grad, _ = sdk.sd_rope_axes(g, None, pos, inv, axes)
    d = torch.randn(y.shape, generator=torch.Generator().manual_seed(14)).to(cuda)
    moved, _ = sdk.sd_rope_axes(d, None, pos, f, axes)  # the rotation is linear: its difference along d
    a, b = (grad.double() * d.double()).sum(), (g.double() * moved.double()).sum()
    assert abs(float(a - b)) <= 2e-6 * float((g.abs() * d.abs()).sum())


def test_infinite_and_nan_values_stay_in_their_head(cuda):
    axes = (32,)
    q = torch.ones(1, 2, 3, 64, device=cuda)
    q[0, 0, 1, 40] = float("inf")  # behind the axis' columns
    q[0, 1, 2, 3] = float("nan")
    pos = torch.arange(2, dtype=torch.int32, device=cuda).view(2, 1)
    y, _ = sdk.sd_rope_axes(q, None, pos, sdk.rope_frequencies(axes), axes)
    assert y[0, 0, 1, 40] == float("inf") and y[0, 0].isfinite().sum() == 3 * 64 - 1
    assert y[0, 1, 2].isnan().sum() == 2 and y[0, 1, :2].isfinite().all()


def test_refusals(cuda):
    axes, f = (64,), sdk.rope_frequencies((64,))
    q = torch.zeros(1, 8, 2, 64, device=cuda)
    pos = torch.zeros(8, 1, dtype=torch.int32, device=cuda)
    with pytest.raises(sdk.SDError, match="overlaps"):
        big = torch.zeros(1, 9, 2, 64, device=cuda)
        sdk.sd_rope_axes(big[:, :8], None, pos, f, axes, q_out=big[:, 1:])
    with pytest.raises(sdk.SDError, match="q_out overlaps k_out"):
        out = torch.zeros_like(q)
        sdk.sd_rope_axes(q, q.clone(), pos, f, axes, q_out=out, k_out=out)
    with pytest.raises(sdk.SDError, match="MISALIGNED"):
        sdk.sd_rope_axes(torch.zeros(1, 8, 2, 65, device=cuda)[..., 1:], None, pos, f, axes)
    with pytest.raises(sdk.SDError, match="heads overlap"):
        sdk.sd_rope_axes(q, None, pos, f, axes, q_out=torch.zeros(1, 8, 1, 64, device=cuda).expand(1, 8, 2, 64))
    assert sdk.sd_rope_axes(q[:, :0], None, pos[:0], f, axes)[0].shape == (1, 0, 2, 64)


def _fused(name, B, L, H, KV, dh, t, dev):
    """(buffer, q, k, layout, the rest): q and k as slices of one buffer that step over one another."""
    g = torch.Generator().manual_seed(31)
    if name == "heads first":  # [B, heads, L, dh]: the batches of q and k alternate
        buf = torch.randn(B, H + 2 * KV, L, dh, generator=g).to(t).to(dev)
        return buf, buf[:, :H], buf[:, H:H + KV], "bhld", buf[:, H + KV:]
    if name == "by head":  # [B, L, heads, 3, dh]: the heads of q and k alternate
        buf = torch.randn(B, L, KV, 3, dh, generator=g).to(t).to(dev)
        return buf, buf[:, :, :, 0], buf[:, :, :, 1], "blhd", buf[:, :, :, 2]
    if name == "by token":  # [L, B, heads, dh], the tokens' rows outermost
        buf = torch.randn(L, B, H + 2 * KV, dh, generator=g).to(t).to(dev)
        x = buf.transpose(0, 1)
        return buf, x[:, :, :H], x[:, :, H:H + KV], "blhd", x[:, :, H + KV:]
    buf = torch.randn(B, L, H + KV, 2 * dh, generator=g).to(t).to(dev)  # columns of wider heads
    return buf, buf[:, :, :H, :dh], buf[:, :, H:, dh:], "blhd", torch.cat((buf[:, :, :H, dh:], buf[:, :, H:, :dh]), 2)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B", [1, 3])
@pytest.mark.parametrize("name", ["heads first", "by head", "by token", "wide heads"])
def test_in_place_on_slices_of_one_buffer(cuda, name, B, dtype):
    axes, L, H, KV, dh = (16, 24, 24), 21, 4, 2, 64
    buf, q, k, layout, rest = _fused(name, B, L, H, KV, dh, TYPES[dtype], cuda)
    pos = torch.randint(0, 64, (B, L, 3), generator=torch.Generator().manual_seed(32), dtype=torch.int32).to(cuda)
    freqs = sdk.rope_frequencies(axes)
    before = rest.clone()
    qo, ko = sdk.sd_rope_axes(q, k, pos, freqs, axes, layout=layout)
    first = (lambda x: x) if layout == "blhd" else (lambda x: x.transpose(1, 2))
    _check(first(qo), first(q), pos, freqs, axes, False, None)
    _check(first(ko), first(k), pos, freqs, axes, False, None)
    sdk.sd_rope_axes(q, k, pos, freqs, axes, layout=layout, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    buf2, q2, k2, _, rest2 = _fused(name, B, L, H, KV, dh, TYPES[dtype], cuda)
    assert torch.equal(before, rest2)
    q2.copy_(qo), k2.copy_(ko)
    assert torch.equal(buf, buf2)  # nothing else was written
