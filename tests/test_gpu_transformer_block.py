"""The transformer-block operators run together, as a block calls them, around torch's projections: residual
and norm, q k v in the rows of one projection, rotary positions in place, masked attention, the output
projection, residual and norm into e4m3. Each operator is checked on the inputs that it got, with the
tolerances of its own tests (see test_gpu_rms_norm.py, test_gpu_rope_axes.py, test_gpu_attention_masked.py)."""
import numpy as np
import pytest
import torch

import oracle
import unet_latent_attention_b200 as sdk

pytestmark = pytest.mark.gpu

H, KV, DH, C, AXES = 6, 3, 64, 320, (16, 24, 24)
BF16 = 2.0 ** -8
ARITH = 100 * 2.0 ** -24


def _f64(t):
    return t.detach().double().cpu().numpy()


class Block:
    """Weights and buffers of one block; ``run`` is the call sequence of a denoising step or a decoder."""

    def __init__(self, dev, seed):
        g = torch.Generator().manual_seed(seed)
        t = lambda *s, m=1.0: (m * torch.randn(*s, generator=g)).to(torch.bfloat16).to(dev)  # noqa: E731
        self.w_qkv, self.w_out = t(C, (H + 2 * KV) * DH, m=C ** -0.5), t(H * DH, C, m=(H * DH) ** -0.5)
        self.n1, self.n2 = 1 + t(C, m=0.1), 1 + t(C, m=0.1)
        self.qn, self.kn = (1 + 0.1 * torch.randn(DH, generator=g)).to(dev), (1 + 0.1 * torch.randn(DH, generator=g)).to(dev)
        self.freqs = sdk.rope_frequencies(AXES)

    def run(self, x, residual, pos, **masks):
        B, L, _ = x.shape
        y, r1 = sdk.sd_rms_norm(x, self.n1, residual=residual)
        rows = (y.view(B * L, C) @ self.w_qkv).view(B, L, H + 2 * KV, DH)
        before = rows.clone()
        q, k, v = rows[:, :, :H], rows[:, :, H:H + KV], rows[:, :, H + KV:]
        sdk.sd_rope_axes(q, k, pos, self.freqs, AXES, q_weight=self.qn, k_weight=self.kn, q_out=q, k_out=k)
        o = sdk.sd_attention_masked(q, k, v, layout="blhd", **masks)
        z = (o.reshape(B * L, H * DH) @ self.w_out).view(B, L, C)
        f8, scales, r2 = sdk.sd_rms_norm_fp8(z, self.n2, residual=r1, block=64)
        return dict(y=y, r1=r1, before=before, q=q, k=k, v=v, o=o, z=z, f8=f8, scales=scales, r2=r2)

    def check(self, s, x, residual, pos, **masks):
        n = lambda t: _f64(t).reshape(-1, t.shape[-1])  # noqa: E731
        ref, h = oracle.rms_norm(n(x), _f64(self.n1), 1e-6, n(residual))
        assert (np.abs(n(s["y"]) - ref) <= np.abs(ref) * (BF16 + ARITH)).all() and (np.abs(n(s["r1"]) - h) <= np.abs(h) * (BF16 + ARITH)).all()
        for name, a, b, w in (("q", 0, H, self.qn), ("k", H, H + KV, self.kn)):
            t = s["before"][:, :, a:b]
            ref = oracle.rope_axes(_f64(t), pos.cpu().numpy(), self.freqs.tolist(), AXES, False, _f64(w))
            top = np.abs(oracle.rms_norm(n(t), _f64(w), 1e-6)[0]).reshape(ref.shape).max(-1, keepdims=True)
            assert (np.abs(_f64(s[name]) - ref) <= np.abs(ref) * BF16 + 2e-6 * top).all()
        assert torch.equal(s["v"], s["before"][:, :, H + KV:])
        first = lambda t: t.transpose(1, 2)  # noqa: E731
        host = {m: (t.cpu().numpy() if torch.is_tensor(t) and t.dtype == torch.int32 else t) for m, t in masks.items()}
        ref, a = oracle.attention_masked(first(s["q"]), first(s["k"]), first(s["v"]), **host)
        assert (np.abs(_f64(first(s["o"])) - ref) <= (BF16 + 4e-4) * a * (1 + BF16) + BF16 * np.abs(ref) + 1e-30).all()
        ref, h = oracle.rms_norm(n(s["z"]), _f64(self.n2), 1e-6, n(s["r1"]))
        assert (np.abs(n(s["r2"]) - h) <= np.abs(h) * (BF16 + ARITH)).all()
        sc = oracle.block_scales(ref, 64)
        assert (np.abs(n(s["scales"]) - sc) <= 2 * ARITH * sc).all()
        c = ref / oracle.spread_scales(sc, C, 64)
        assert (np.abs(n(s["f8"].float()) - c) <= np.maximum(2.0 ** -4 * np.abs(c), 2.0 ** -10) + 3 * ARITH * np.abs(c)).all()


def _case(name, dev):
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if name == "images":  # three packed images with their prompts, the rows behind them unused
        return 1, 300, dict(q_offsets=ints(0, 90, 91, 277), k_offsets=ints(0, 90, 91, 277))
    if name == "text":  # padded prompts with a bias by distance
        bias = torch.randn(H, 2 * 16 + 1, generator=torch.Generator().manual_seed(2)).to(dev)
        return 3, 77, dict(kv_lens=ints(77, 5, 40), bias=bias)
    return 2, 200, dict(causal=True, prefix_lens=ints(77, 3), cap=20.0)  # image tokens behind a prompt


@pytest.mark.parametrize("name", ["images", "text", "raster"])
def test_block(cuda, name):
    B, L, masks = _case(name, cuda)
    g = torch.Generator().manual_seed(5)
    x, r = ((m * torch.randn(B, L, C, generator=g)).to(torch.bfloat16).to(cuda) for m in (1.0, 3.0))
    pos = torch.randint(0, 64, (B, L, 3), generator=g, dtype=torch.int32).to(cuda)
    block = Block(cuda, 3)
    s = block.run(x, r, pos, **masks)
    sdk.sd_device_status()
    block.check(s, x, r, pos, **masks)


def test_blocks_captured_and_replayed_on_new_inputs(cuda):
    B, L, masks = _case("raster", cuda)
    g = torch.Generator().manual_seed(6)
    make = lambda: tuple((m * torch.randn(B, L, C, generator=g)).to(torch.bfloat16).to(cuda) for m in (1.0, 3.0))  # noqa: E731
    x, r = make()
    pos = torch.randint(0, 64, (B, L, 3), generator=g, dtype=torch.int32).to(cuda)
    block = Block(cuda, 4)
    block.run(x, r, pos, **masks)  # loads the kernels and torch's workspaces
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        s = block.run(x, r, pos, **masks)
    for _ in range(2):
        x2, r2 = make()
        x.copy_(x2)
        r.copy_(r2)
        graph.replay()
        torch.cuda.synchronize()
        sdk.sd_device_status()
        block.check(s, x, r, pos, **masks)


def test_a_token_at_a_time_is_the_whole_sequence(cuda):
    # decoding against a cache gives what the causal call over the sequence gives, position by position
    B, L = 2, 40
    g = torch.Generator().manual_seed(7)
    q, k, v = (torch.randn(B, L, h, DH, generator=g).to(torch.bfloat16).to(cuda) for h in (H, KV, KV))
    pos = torch.arange(L, dtype=torch.int32, device=cuda).view(L, 1)
    f = sdk.rope_frequencies((DH,))
    qr, kr = sdk.sd_rope_axes(q, k, pos, f, (DH,), pairs="half")
    whole = sdk.sd_attention_masked(qr, kr, v, layout="blhd", causal=True)
    cache_k, cache_v = (torch.full((B, 64, KV, DH), float("nan"), dtype=torch.bfloat16, device=cuda) for _ in range(2))
    for i in range(L):
        qi, ki = sdk.sd_rope_axes(q[:, i:i + 1], k[:, i:i + 1], pos[i:i + 1], f, (DH,), pairs="half")
        assert torch.equal(qi, qr[:, i:i + 1]) and torch.equal(ki, kr[:, i:i + 1])
        cache_k[:, i:i + 1], cache_v[:, i:i + 1] = ki, v[:, i:i + 1]
        n = torch.full((B,), i + 1, dtype=torch.int32, device=cuda)
        o = sdk.sd_attention_masked(qi, cache_k, cache_v, layout="blhd", causal=True, kv_lens=n, q_starts=n - 1)
        a = sdk.sd_attention_masked(qi, kr[:, :i + 1].contiguous(), v[:, :i + 1].abs().contiguous(), layout="blhd").float()
        # both round each weight and the output: twice the tolerance of one
        assert ((o.float() - whole[:, i:i + 1].float()).abs() <= 4 * BF16 * (a * 1.01) + 1e-6).all()


def test_offsets_beyond_32_bits(cuda):
    # rows, batches and caches whose elements lie more than 2^32 apart, in one large buffer
    far = (1 << 32) + 4096
    big = torch.empty(far + (1 << 20), dtype=torch.bfloat16, device=cuda)
    g = torch.Generator().manual_seed(8)

    def spread(at, *shape):  # [2, ...], the second one `far` elements behind the first
        n = int(np.prod(shape))
        strides = [int(np.prod(shape[i + 1:])) for i in range(len(shape))]
        x = big.as_strided((2, *shape), (far, *strides), at)
        dense = torch.randn(2, *shape, generator=g).to(torch.bfloat16).to(cuda)
        x.copy_(dense)
        return x, dense, at + n

    x, xd, at = spread(0, 1280)
    out, _, at = spread(at, 1280)
    w = 1 + 0.1 * torch.randn(1280, generator=g).to(cuda)
    sdk.sd_rms_norm(x, w, out=out)
    assert torch.equal(out, sdk.sd_rms_norm(xd, w))
    q, qd, at = spread(at, 5, H, DH)
    k, kd, at = spread(at, 300, KV, DH)
    v, vd, at = spread(at, 300, KV, DH)
    o = torch.empty(far + 5 * H * DH, dtype=torch.bfloat16, device=cuda).as_strided((2, 5, H, DH), (far, H * DH, DH, 1))
    pos = torch.randint(0, 64, (2, 5, 3), generator=g, dtype=torch.int32).to(cuda)
    f = sdk.rope_frequencies(AXES)
    qo, ko = sdk.sd_rope_axes(qd, kd[:, :5], pos, f, AXES)
    sdk.sd_rope_axes(q, k[:, :5], pos, f, AXES, q_out=q, k_out=k[:, :5])
    assert torch.equal(q, qo) and torch.equal(k[:, :5], ko) and torch.equal(k[:, 5:], kd[:, 5:])
    vd[:, 290, 1, 3] = float("inf")  # found again in v itself by the rows that see it
    v.copy_(vd)
    n = torch.tensor([295, 300], dtype=torch.int32, device=cuda)
    sdk.sd_attention_masked(q, k, v, layout="blhd", causal=True, kv_lens=n, q_starts=n - 5, out=o)
    want = sdk.sd_attention_masked(qo, torch.cat((ko, kd[:, 5:]), 1), vd, layout="blhd", causal=True, kv_lens=n, q_starts=n - 5)
    sdk.sd_device_status()
    assert torch.equal(o, want) and want.isinf().any() and not want.isnan().any()
