"""GPU parity of sd_attention_masked where scores are large, infinite or at the ends of their type.

Products q.k are small integers (or 2^20 and small integers), so the tensor cores' fp32 sums hold them exactly
and both sides have the same ties. What is left of a weight's error: ex2.approx (2^-22 relative), the
difference from the maximum and its product with the scale (2^-23 |x| at a weight of 2^-x: below 1e-7), the
rounded product of a maximum of up to 2^16 (half a step, 2^-8 * ln 2, for the keys before a raise of the
maximum, whose weights are below 2^-8 by then: 1.1e-5) and sums of at most 64 dependent terms (64 * 2^-24 =
4e-6). ARITH = 5e-5 is above them together, for the numerator and for the denominator; the weights are rounded
to the inputs' type (half a step u), fp16 weights below 2^-14 to 2^-25, and the output once more. A cap's tanh is
off by 2e-7 of the score, or of the cap where the score is above half of it: below 2e-5 at a cap of 30 or at
scores of up to 60 and larger caps."""
import numpy as np
import pytest
import torch

import oracle
import unet_latent_attention_b200 as sdk

pytestmark = pytest.mark.gpu

ARITH = 5e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _whole_numbers(B, H, KV, Lq, Lk, dh, t, seed, dev):
    """q and k of whole numbers from -3 to 3 (|q.k| <= 9 dh), normal v."""
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randint(-3, 4, s, generator=g).float() for s in ((B, H, Lq, dh), (B, KV, Lk, dh)))
    v = torch.randn(B, KV, Lk, dh, generator=g)
    return tuple(x.to(t).to(dev) for x in (q, k, v))


def _check(o, q, k, v, **kw):
    sdk.sd_device_status()
    host = {n: (x.cpu().numpy() if torch.is_tensor(x) and x.dtype == torch.int32 else x) for n, x in kw.items()}
    ref, a = oracle.attention_masked(q, k, v, **host)
    got = o.double().cpu().numpy()
    u = torch.finfo(q.dtype).eps / 2
    tiny = 2.0 ** -25 * np.abs(v.double().cpu().numpy()).sum(axis=2).max() if q.dtype == torch.float16 else 0.0
    assert np.isfinite(got).all()
    tol = (u + 2 * ARITH) * a * (1 + u) + u * np.abs(ref) + tiny + 1e-30
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) - tol).max())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("scale", [100.0, 1e5, 1e9, 1e30, 3e38])
@pytest.mark.parametrize("dh", [64, 128, 160])
def test_large_scales(cuda, dh, scale, dtype):
    # a row's largest score has the weight 1 (shared by its ties), however large the score is
    B, H, KV, Lq, Lk = 2, 4, 2, 200, 333
    q, k, v = _whole_numbers(B, H, KV, Lq, Lk, dh, TYPES[dtype], dh, cuda)
    lens, prefix = _ints([333, 150], cuda), _ints([0, 77], cuda)
    for kw in (dict(), dict(causal=True), dict(kv_lens=lens), dict(causal=True, kv_lens=lens, prefix_lens=prefix)):
        kw = dict(kw, scale=scale)
        _check(sdk.sd_attention_masked(q, k, v, **kw), q, k, v, **kw)
    if scale < 1e37:  # with a bias the score itself has to stay in fp32
        for R in (0, 5):  # one value a head: it moves no tie; tiles beyond the table and across it
            bias = torch.tensor([0.5, -2.0, 7.0, 0.0], device=cuda)[:, None].expand(H, 2 * R + 1).contiguous()
            kw = dict(bias=bias, causal=True, scale=scale)
            _check(sdk.sd_attention_masked(q, k, v, **kw), q, k, v, **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("scale", [1e9, 3e38])
def test_large_scales_of_few_queries_and_documents(cuda, scale, dtype):
    # keys split over a cluster, whose parts have maxima of their own
    q, k, v = _whole_numbers(2, 4, 2, 1, 4000, 128, TYPES[dtype], 5, cuda)
    for kw in (dict(), dict(kv_lens=_ints([4000, 900], cuda))):
        kw = dict(kw, scale=scale)
        _check(sdk.sd_attention_masked(q, k, v, **kw), q, k, v, **kw)
    q, k, v = _whole_numbers(1, 2, 2, 300, 300, 64, TYPES[dtype], 6, cuda)
    off = _ints([0, 70, 71, 290], cuda)
    kw = dict(q_offsets=off, k_offsets=off, scale=scale)
    _check(sdk.sd_attention_masked(q, k, v, **kw), q, k, v, **kw)
    if scale < 1e37:
        kw.update(k_offsets=_ints([0, 100, 120, 300], cuda), bias=torch.full((2, 9), 3.0, device=cuda))  # different shifts in one tile
        _check(sdk.sd_attention_masked(q, k, v, **kw), q, k, v, **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("Lq,Lk", [(200, 333), (1, 3000)])
def test_scores_around_a_large_value(cuda, Lq, Lk, sign, dtype):
    # q.k = +-2^20 + a small whole number: an ordinary softmax around +-2^17, and a flat one around +-2^13
    q, k, v = _whole_numbers(1, 2, 2, Lq, Lk, 64, TYPES[dtype], 7, cuda)
    q[..., 0], k[..., 0] = 1024.0, sign * 1024.0
    for kw in (dict(scale=0.125), dict(scale=0.125, causal=True), dict(scale=0.0078125, causal=True)):
        _check(sdk.sd_attention_masked(q, k, v, **kw), q, k, v, **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_a_large_score_in_one_row(cuda, dtype):
    # its neighbours keep their bits, and a tile of large scores after one of small ones takes over
    q, k, v = _whole_numbers(1, 2, 2, 150, 400, 64, TYPES[dtype], 8, cuda)
    want = sdk.sd_attention_masked(q, k, v, scale=0.125)
    q2 = q.clone()
    q2[:, :, 40] = 2.0 ** 14 * q[:, :, 40]
    o = sdk.sd_attention_masked(q2, k, v, scale=1e3)
    _check(o, q2, k, v, scale=1e3)
    o = sdk.sd_attention_masked(q2, k, v, scale=0.125)
    rest = [i for i in range(150) if i != 40]
    assert torch.equal(o[:, :, rest], want[:, :, rest])
    _check(o, q2, k, v, scale=0.125)
    k2 = k.clone()
    k2[:, :, 256:] = 2.0 ** 13 * k[:, :, 256:]
    _check(sdk.sd_attention_masked(q, k2, v, scale=1e4), q, k2, v, scale=1e4)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cap", [30.0, 1e4, 1e6])
@pytest.mark.parametrize("dh", [64, 128])
def test_capped_scores_do_not_depend_on_other_scores(cuda, dh, cap, dtype):
    # beside a score above half the cap, of an unseen key or of another row, all others keep their bits
    t = TYPES[dtype]
    q, k, v = _whole_numbers(2, 2, 2, 150, 400, dh, t, 9 + dh, cuda)
    for kw in (dict(kv_lens=_ints([390, 140], cuda)), dict(kv_lens=_ints([390, 140], cuda), bias=torch.randn(2, 9, generator=torch.Generator().manual_seed(1)).to(cuda))):
        kw = dict(kw, cap=cap)
        want = sdk.sd_attention_masked(q, k, v, **kw)
        _check(want, q, k, v, **kw)
        for x in (float("nan"), float("inf"), float("-inf"), torch.finfo(t).max):
            k2 = k.clone()
            k2[0, :, 390:], k2[1, :, 140:] = x, x
            assert torch.equal(sdk.sd_attention_masked(q, k2, v, **kw), want), x
        q2 = q.clone()
        q2[:, :, 40] = torch.where(q[:, :, 40] < 0, -60000.0, 60000.0)
        rest = [i for i in range(150) if i != 40]
        assert torch.equal(sdk.sd_attention_masked(q2, k, v, **kw)[:, :, rest], want[:, :, rest])
    want = sdk.sd_attention_masked(q, k, v, causal=True, cap=cap)
    k2 = k.clone()
    k2[:, :, 300] = torch.finfo(t).max  # the last 50 rows see it
    assert torch.equal(sdk.sd_attention_masked(q, k2, v, causal=True, cap=cap)[:, :, :50], want[:, :, :50])
    q, k, v = _whole_numbers(2, 2, 2, 1, 3000, dh, t, 10 + dh, cuda)  # keys split over a cluster
    kw = dict(cap=cap, kv_lens=_ints([2990, 700], cuda))
    want = sdk.sd_attention_masked(q, k, v, **kw)
    k[0, :, 2990:], k[1, :, 700:] = float("nan"), torch.finfo(t).max
    assert torch.equal(sdk.sd_attention_masked(q, k, v, **kw), want)


def test_a_large_cap_of_large_scores(cuda):
    # q.k = 2^66 * a whole number (its square is beyond fp32) under a cap of 1e30: as if there were no cap
    for Lq, Lk in ((150, 333), (1, 3000)):
        q, k, v = _whole_numbers(1, 2, 2, Lq, Lk, 64, torch.bfloat16, 11, cuda)
        q, k = q * 2.0 ** 33, k * 2.0 ** 33
        for kw in (dict(), dict(causal=True), dict(bias=torch.full((2, 9), 3.0, device=cuda))):
            kw = dict(kw, cap=1e30)
            _check(sdk.sd_attention_masked(q, k, v, **kw), q, k, v, **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("ahead", [20.0, -20.0])
@pytest.mark.parametrize("cap", [30.0, 1e4, 1e6, 1e7])
def test_the_cap_of_scores_of_its_size(cuda, cap, ahead, dtype):
    # Two keys with scores of 0.45 and 0.225 of the cap, which a bias leaves 20 apart: the one ahead has all the
    # weight. A score is off by 2e-7 of the cap and the bias by half a step of it: at 1e7 3 together.
    t = TYPES[dtype]
    q, k = torch.zeros(1, 1, 1, 64, dtype=t, device=cuda), torch.zeros(1, 1, 2, 64, dtype=t, device=cuda)
    q[..., 0], k[0, 0, 0, 0], k[0, 0, 1, 0] = 4800.0, 12032.0, 6016.0
    scale = cap * 0.45 / (4800.0 * 12032.0)
    v = torch.randn(1, 1, 2, 64, generator=torch.Generator().manual_seed(12)).to(t).to(cuda)
    apart = cap * (np.tanh(0.45) - np.tanh(0.225))
    bias = torch.tensor([[-apart + ahead, 0.0, 0.0]], dtype=torch.float32, device=cuda)
    o = sdk.sd_attention_masked(q, k, v, scale=scale, cap=cap, bias=bias)
    sdk.sd_device_status()
    assert torch.equal(o[0, 0, 0], v[0, 0, 0 if ahead > 0 else 1])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("Lq,Lk", [(150, 150), (2, 2000)])
def test_rows_of_minus_infinity_are_zero_beside_infinite_values(cuda, Lq, Lk, dtype):
    # the last row sees keys with a bias of -infinity only, one of them with an infinite and a NaN value
    q, k, v = _whole_numbers(1, 2, 2, Lq, Lk, 64, TYPES[dtype], 13, cuda)
    d = torch.arange(-Lk, Lk + 1, device=cuda)
    bias = torch.where(d == Lk - Lq + 1, 0.0, float("-inf")).expand(2, -1).contiguous()  # key i + 1 + Lk - Lq of row i
    starts = _ints([0], cuda)
    want = sdk.sd_attention_masked(q, k, v, bias=bias, q_starts=starts)
    v[:, :, Lk - 3, 3], v[:, :, Lk - 3, 5] = float("inf"), float("nan")
    o = sdk.sd_attention_masked(q, k, v, bias=bias, q_starts=starts)
    sdk.sd_device_status()
    assert (want[:, :, -1] == 0).all() and (o[:, :, -1] == 0).all()
    fine = [c for c in range(64) if c not in (3, 5)]
    assert torch.equal(o[..., fine], want[..., fine])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dh", [8, 40, 64, 80, 128, 160])
@pytest.mark.parametrize("Lq,Lk", [(1, 1), (5, 2050), (200, 333)])
def test_ordinary_scores(cuda, dh, Lq, Lk, dtype):
    # with exact products nothing but the weights' own roundings is left
    q, k, v = _whole_numbers(2, 4, 2, Lq, Lk, dh, TYPES[dtype], 14 + dh, cuda)
    lens, starts = _ints([Lk, Lk // 3], cuda), _ints([Lk - Lq, 0], cuda)
    bias = torch.randn(4, 61, generator=torch.Generator().manual_seed(15)).to(cuda)
    for kw in (dict(), dict(causal=True, kv_lens=lens, q_starts=starts), dict(cap=30.0, kv_lens=lens), dict(bias=bias), dict(bias=bias, cap=9.0, causal=True)):
        _check(sdk.sd_attention_masked(q, k, v, **kw), q, k, v, **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("scale", [0.125, 1e9])
@pytest.mark.parametrize("Lq,Lk", [(150, 400), (1, 3000)])
def test_large_scores_beside_unseen_values(cuda, Lq, Lk, scale, dtype):
    # infinities and NaN behind the lengths, and seen keys with a score of -infinity, whatever form the row takes
    t = TYPES[dtype]
    for dh in (64, 128):
        q, k, v = _whole_numbers(2, 4, 2, Lq, Lk, dh, t, 16 + dh, cuda)
        lens = _ints([Lk - 10, Lk // 3], cuda)
        for kw in (dict(), dict(bias=torch.full((4, 5), -2.0, device=cuda))):
            kw = dict(kw, scale=scale, kv_lens=lens)
            want = sdk.sd_attention_masked(q, k, v, **kw)
            _check(want, q, k, v, **kw)
            for x in (float("nan"), float("inf"), float("-inf"), torch.finfo(t).max):
                k2, v2 = k.clone(), v.clone()
                for b, n in enumerate(lens.tolist()):
                    k2[b, :, n:], v2[b, :, n:] = x, x
                assert torch.equal(sdk.sd_attention_masked(q, k2, v2, **kw), want), x
        bias = torch.full((4, 2 * Lk + 1), 0.0, device=cuda)
        bias[:, ::3] = float("-inf")
        kw = dict(scale=scale, kv_lens=lens, bias=bias)
        _check(sdk.sd_attention_masked(q, k, v, **kw), q, k, v, **kw)
