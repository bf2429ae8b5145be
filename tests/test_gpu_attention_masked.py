"""GPU parity of sd_attention_masked against the fp64 oracle.

Tolerance. Each weight is rounded once to the inputs' type (half a step u: 2^-8 bf16, 2^-11 fp16) and carries
the errors of the score and of exp2: scores in fp32 (dh products, |x| < 64 in units of log2: 64 * 2^-24 * ln 2
< 3e-6), a cap's tanh (a few 2^-23 of cap * log2(e) < 100: 5e-5) and the polynomial exp2 (7.5e-5). With
ARITH = 2e-4 for all of these together, numerator and denominator are off by at most (u + ARITH) A with
A = sum_j p_j |v_j| and by ARITH |o| <= ARITH A; fp16 weights below 2^-14 add half their step of 2^-24 each, times |v_j|, over a
sum of at least 1. The output is rounded once more (u |o|, on a value that is off itself)."""
import numpy as np
import pytest
import torch

import oracle
import unet_latent_attention_b200 as sdk

pytestmark = pytest.mark.gpu

ARITH = 2e-4
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _tensors(B, H, KV, Lq, Lk, dh, t, seed, dev, blhd=False):
    g = torch.Generator().manual_seed(seed)
    shapes = [(B, H, Lq, dh), (B, KV, Lk, dh), (B, KV, Lk, dh)]
    q, k, v = (torch.randn(s, generator=g) * m for s, m in zip(shapes, (1.5, 1.0, 1.0)))
    q, k, v = (x.to(t).to(dev) for x in (q, k, v))
    return tuple(x.transpose(1, 2).contiguous() for x in (q, k, v)) if blhd else (q, k, v)


def _check(o, q, k, v, layout="bhld", out=None, **kw):
    sdk.sd_device_status()
    first = (lambda x: x) if layout == "bhld" else (lambda x: x.transpose(1, 2))
    host = {n: (x.cpu().numpy() if torch.is_tensor(x) and x.dtype == torch.int32 else x) for n, x in kw.items()}
    ref, a = oracle.attention_masked(first(q), first(k), first(v), out=None if out is None else first(out), **host)
    got = first(o).double().cpu().numpy()
    u = torch.finfo(q.dtype).eps / 2
    tiny = 2.0 ** -25 * np.abs(np.nan_to_num(first(v).double().cpu().numpy(), posinf=0, neginf=0)).sum(axis=2).max() if q.dtype == torch.float16 else 0.0
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isinf(got), np.isinf(ref))
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
    with np.errstate(invalid="ignore"):
        err, tol = np.abs(got - ref), (u + 2 * ARITH) * np.nan_to_num(a, posinf=0) * (1 + u) + u * np.abs(ref) + tiny + 1e-30
    assert (err[fine] <= tol[fine]).all(), float((err - tol)[fine].max())
    return ref


def _ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _bias(H, R, seed, dev):
    return torch.randn(H, 2 * R + 1, generator=torch.Generator().manual_seed(seed)).to(dev)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dh", [8, 40, 64, 72, 80, 128, 136, 160])
@pytest.mark.parametrize("Lq,Lk", [(1, 1), (1, 129), (7, 77), (129, 255), (300, 260), (513, 640)])
def test_causal_and_whole(cuda, dh, Lq, Lk, dtype):
    q, k, v = _tensors(2, 2, 2, Lq, Lk, dh, TYPES[dtype], dh + Lq + Lk, cuda)
    for causal in (False, True):  # more queries than keys: the first see nothing
        _check(sdk.sd_attention_masked(q, k, v, causal=causal), q, k, v, causal=causal)


def test_without_masks_like_sd_attention(cuda):
    q, k, v = _tensors(2, 8, 8, 1024, 1024, 64, torch.bfloat16, 1, cuda)
    a, b = sdk.sd_attention_masked(q, k, v).float(), sdk.sd_attention(q, k, v).float()
    assert (a - b).abs().max() <= 2 * 2.0 ** -8 * b.abs().max()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", ["bhld", "blhd"])
@pytest.mark.parametrize("dh,H,KV", [(64, 4, 2), (80, 3, 1), (128, 6, 6), (160, 4, 1)])
def test_lengths_starts_and_prefixes(cuda, dh, H, KV, layout, dtype):
    Lq, Lk, B = 200, 333, 5
    q, k, v = _tensors(B, H, KV, Lq, Lk, dh, TYPES[dtype], 11 + dh, cuda, layout == "blhd")
    lens, starts, prefix = _ints([333, 0, 1, 200, 999], cuda), _ints([133, -50, 0, 400, -2 ** 31], cuda), _ints([0, 5, 77, 150, 1000], cuda)
    for kw in (dict(kv_lens=lens), dict(causal=True, kv_lens=lens), dict(causal=True, q_starts=starts),
               dict(causal=True, prefix_lens=prefix), dict(causal=True, kv_lens=lens, q_starts=starts, prefix_lens=prefix)):
        _check(sdk.sd_attention_masked(q, k, v, layout=layout, **kw), q, k, v, layout, **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cap", [0.0, 2.0, 30.0])
@pytest.mark.parametrize("dh,R", [(64, None), (64, 0), (64, 16), (80, 300), (128, 40), (160, 1000)])
def test_cap_and_bias(cuda, dh, R, cap, dtype):
    B, H, Lq, Lk = 2, 3, 270, 400
    q, k, v = _tensors(B, H, H, Lq, Lk, dh, TYPES[dtype], 21 + dh, cuda)
    bias = None if R is None else _bias(H, R, 22, cuda)
    for kw in (dict(), dict(causal=True), dict(kv_lens=_ints([400, 100], cuda), q_starts=_ints([7, -3], cuda))):
        kw = dict(kw, cap=cap, bias=bias)
        _check(sdk.sd_attention_masked(q, k, v, **kw), q, k, v, **kw)


def test_cap_of_large_scores(cuda):
    q, k, v = _tensors(1, 2, 2, 130, 140, 64, torch.bfloat16, 23, cuda)
    q = q * 64  # scores of +-500: the tanh saturates
    _check(sdk.sd_attention_masked(q, k, v, cap=5.0), q, k, v, cap=5.0)


OFFSETS = [([0, 100, 100, 400, 421], [0, 100, 100, 400, 421]), ([0, 1, 2, 3, 440], [0, 1, 2, 3, 440]),
           ([5, 130, 300], [17, 20, 430]), ([0, 450], [0, 450]), ([0, 50, 200, 300, 320], [0, 0, 300, 310, 450])]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dh", [64, 80, 160])
@pytest.mark.parametrize("qo,ko", OFFSETS)
def test_documents(cuda, qo, ko, dh, dtype):
    H, T = 2, 450
    q, k, v = _tensors(1, H, 1, T, T, dh, TYPES[dtype], 31 + dh, cuda, True)
    off = dict(q_offsets=_ints(qo, cuda), k_offsets=_ints(ko, cuda))
    for kw in (dict(), dict(causal=True), dict(causal=True, prefix_lens=_ints([20] * (len(qo) - 1), cuda)),
               dict(bias=_bias(H, 30, 32, cuda)), dict(causal=True, cap=20.0, bias=_bias(H, 500, 33, cuda), q_starts=_ints([3] * (len(qo) - 1), cuda))):
        kw = dict(kw, **off)
        out = torch.full_like(q, 7.0)
        o = sdk.sd_attention_masked(q, k, v, layout="blhd", out=out, **kw)
        assert o is out
        _check(o, q, k, v, "blhd", out=torch.full_like(q, 7.0), **kw)
        assert (o[:, qo[-1]:] == 7).all() and (o[:, :qo[0]] == 7).all()
    o = sdk.sd_attention_masked(q, k, v, layout="blhd", **off)
    assert (o[:, qo[-1]:] == 0).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,H,KV,Lq,Lk,dh", [(1, 1, 1, 1, 5000, 64), (2, 8, 2, 1, 4097, 128), (3, 4, 4, 2, 2000, 40), (1, 16, 1, 5, 3001, 160),
                                             (2, 6, 2, 3, 1500, 80), (1, 12, 12, 70, 1111, 64)])
def test_few_queries_split_over_a_cluster(cuda, B, H, KV, Lq, Lk, dh, dtype):
    q, k, v = _tensors(B, H, KV, Lq, Lk, dh, TYPES[dtype], 41 + dh, cuda, True)
    lens = [Lk, Lk // 3, 0][:B]
    starts = _ints([n - Lq for n in lens], cuda)
    bias = _bias(H, 100, 42, cuda)
    for kw in (dict(), dict(causal=True, kv_lens=_ints(lens, cuda), q_starts=starts), dict(bias=bias, cap=15.0, q_starts=starts)):
        o = sdk.sd_attention_masked(q, k, v, layout="blhd", **kw)
        _check(o, q, k, v, "blhd", **kw)
        for _ in range(3):  # the join's order is fixed
            assert torch.equal(o, sdk.sd_attention_masked(q, k, v, layout="blhd", **kw))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dh", [64, 80, 160])
def test_values_of_unseen_keys_never_matter(cuda, dh, dtype):
    t = TYPES[dtype]
    bad = [float("nan"), float("inf"), float("-inf"), torch.finfo(t).max]
    q, k, v = _tensors(2, 2, 2, 300, 300, dh, t, 51 + dh, cuda)
    lens = _ints([290, 140], cuda)
    kw = dict(kv_lens=lens)
    want = sdk.sd_attention_masked(q, k, v, **kw)
    for x in bad:  # behind the lengths
        k2, v2 = k.clone(), v.clone()
        for b, n in enumerate((290, 140)):
            k2[b, :, n:], v2[b, :, n:] = x, x
        assert torch.equal(sdk.sd_attention_masked(q, k2, v2, **kw), want), x
    want = sdk.sd_attention_masked(q, k, v, causal=True)
    for x in bad:  # later keys: rows before them keep their bits, rows from them on get the value
        k2, v2 = k.clone(), v.clone()
        v2[:, :, 200, 3] = x
        o = sdk.sd_attention_masked(q, k2, v2, causal=True)
        assert torch.equal(o[:, :, :200], want[:, :, :200]), x
        if x != torch.finfo(t).max:
            _check(o, q, k2, v2, causal=True)
        k2[:, :, 200] = x
        assert torch.equal(sdk.sd_attention_masked(q, k2, v2, causal=True)[:, :, :200], want[:, :, :200]), x
    # a document of NaN beside another in the same tiles
    off = dict(q_offsets=_ints([0, 130, 300], cuda), k_offsets=_ints([0, 130, 300], cuda))
    want = sdk.sd_attention_masked(q[:1], k[:1], v[:1], **off)
    for x in bad[:3]:
        q2, k2, v2 = q[:1].clone(), k[:1].clone(), v[:1].clone()
        k2[:, :, :130], v2[:, :, :130], q2[:, :, :130] = x, x, x
        o = sdk.sd_attention_masked(q2, k2, v2, **off)
        assert torch.equal(o[:, :, 130:], want[:, :, 130:]) and o[:, :, :130].isnan().all()
    # few queries, keys split over a cluster
    q1 = q[:, :, :1].contiguous()
    kk, vv = (torch.cat([x] * 8, 2) for x in (k, v))
    kw = dict(kv_lens=_ints([2000, 700], cuda))
    want = sdk.sd_attention_masked(q1, kk, vv, **kw)
    for x in bad:
        k2, v2 = kk.clone(), vv.clone()
        for b, n in enumerate((2000, 700)):
            k2[b, :, n:], v2[b, :, n:] = x, x
        assert torch.equal(sdk.sd_attention_masked(q1, k2, v2, **kw), want), x
        v2[:, :, 699, 1] = x  # seen by both, in a masked tile of the second
        if x != torch.finfo(t).max:
            _check(sdk.sd_attention_masked(q1, k2, v2, **kw), q1, k2, v2, **kw)


def test_biases_of_minus_infinity_and_of_the_lowest_value(cuda):
    B, H, L, R = 1, 2, 300, 299
    q, k, v = _tensors(B, H, H, L, L, 64, torch.bfloat16, 61, cuda)
    d = torch.arange(-R, R + 1, device=cuda)
    window = torch.where(d.abs() <= 20, 0.0, float("-inf")).expand(H, -1).contiguous()  # a band: tiles that no row sees
    _check(sdk.sd_attention_masked(q, k, v, bias=window), q, k, v, bias=window)
    window = torch.where(d > 150, 0.0, float("-inf")).expand(H, -1).contiguous()  # the last rows see nothing: 0
    o = sdk.sd_attention_masked(q, k, v, bias=window)
    assert (o[:, :, 149:] == 0).all()
    _check(o, q, k, v, bias=window)
    for low in (torch.finfo(torch.float32).min, float(torch.finfo(torch.bfloat16).min), -65504.0):
        window = torch.where(d > 150, 0.0, low).expand(H, -1).contiguous()
        o = sdk.sd_attention_masked(q, k, v, bias=window)
        if low == -65504.0:  # near it fp32 holds scores to 2^-8 only: the rows of nothing else are left out
            o, qq, kk = o[:, :, :149], q[:, :, :149], k
            ref, a = oracle.attention_masked(q, k, v, bias=window)
            assert (np.abs(o.double().cpu().numpy() - ref[:, :, :149]) <= (2 * 2.0 ** -8 + 2 * ARITH) * a[:, :, :149]).all()
        else:  # every score is the lowest value: the mean of the keys
            _check(o, q, k, v, bias=window)


@pytest.mark.parametrize("R", [0, 1, 40])
def test_lowest_bias_over_whole_tiles(cuda, R):
    # tiles whose distances all lie beyond the table: its ends hold -infinity, the lowest value or a large one
    q, k, v = _tensors(1, 2, 2, 300, 700, 64, torch.bfloat16, 63 + R, cuda)
    for low in (float("-inf"), torch.finfo(torch.float32).min, float(torch.finfo(torch.bfloat16).min), -1e20, -3.0, 2.5):
        bias = torch.zeros(2, 2 * R + 1, device=cuda)
        bias[:, 0] = bias[:, -1] = low
        _check(sdk.sd_attention_masked(q, k, v, bias=bias), q, k, v, bias=bias)
        kw = dict(bias=bias, q_starts=_ints([-200], cuda), causal=False)
        _check(sdk.sd_attention_masked(q, k, v, **kw), q, k, v, **kw)


def test_strided_views_and_more_keys_than_heads_share(cuda):
    # q, k, v in the rows of one projection, the output in a wider buffer
    B, L, H, KV, dh = 2, 150, 4, 2, 64
    g = torch.Generator().manual_seed(71)
    rows = torch.randn(B, L, H + 2 * KV, dh, generator=g).to(torch.bfloat16).to(cuda)
    q, k, v = rows[:, :, :H], rows[:, :, H:H + KV], rows[:, :, H + KV:]
    wide = torch.full((B, L, H + 3, dh), 3.0, dtype=torch.bfloat16, device=cuda)
    o = sdk.sd_attention_masked(q, k, v, layout="blhd", causal=True, out=wide[:, :, 1:H + 1])
    _check(o, q, k, v, "blhd", causal=True)
    assert (wide[:, :, 0] == 3).all() and (wide[:, :, H + 1:] == 3).all()
    # every other token, a batch of one out of a longer cache
    cache = torch.randn(1, 400, KV, dh, generator=g).to(torch.bfloat16).to(cuda)
    k2, v2 = cache[:, ::2], cache[:, 1::2]
    _check(sdk.sd_attention_masked(q[:1], k2, v2, layout="blhd"), q[:1], k2, v2, "blhd")


def test_many_query_tiles(cuda):
    # more pairs of query tiles than SMs, causal and not, rows checked one by one
    H, L, dh = 20, 2100, 64
    q, k, v = _tensors(1, H, H, L, L, dh, torch.bfloat16, 81, cuda)
    for causal in (False, True):
        o = sdk.sd_attention_masked(q, k, v, causal=causal)
        sdk.sd_device_status()
        for i in (0, 1, 127, 128, 255, 256, 1023, 2047, 2048, 2099):
            n = i + 1 if causal else L
            ref, a = oracle.attention_masked(q[:, :, i:i + 1], k[:, :, :n], v[:, :, :n])
            err = np.abs(o[:, :, i:i + 1].double().cpu().numpy() - ref)
            assert (err <= (2.0 ** -8 + 2 * ARITH) * a * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)).all(), (causal, i)


@pytest.mark.parametrize("dh,H", [(64, 20), (80, 20), (160, 10)])
@pytest.mark.parametrize("offsets", [[0, 100, 2100], [0, 2000, 2100], [0, 128, 256, 1500, 2050], [0, 1000, 1001, 2040]])
def test_many_query_tiles_of_documents(cuda, offsets, dh, H):
    # the two query tiles of a CTA end their keys far apart: neither may hold the other's up
    L = 2100
    q, k, v = _tensors(1, H, H, L, L, dh, torch.bfloat16, 83 + dh, cuda)
    off = _ints(offsets, cuda)
    for causal in (False, True):
        o = sdk.sd_attention_masked(q, k, v, causal=causal, q_offsets=off, k_offsets=off)
        sdk.sd_device_status()
        for i in sorted({0, 127, 128, 255, 256, L - 1, *(x for d in offsets for x in (d - 1, d) if 0 <= x < L)}):
            d = max(x for x in offsets if x <= i)
            e = next((x for x in offsets if x > i), None)
            if e is None:
                assert (o[:, :, i] == 0).all()
                continue
            ref, a = oracle.attention_masked(q[:, :, i:i + 1], k[:, :, d:i + 1 if causal else e], v[:, :, d:i + 1 if causal else e])
            err = np.abs(o[:, :, i:i + 1].double().cpu().numpy() - ref)
            assert (err <= (2.0 ** -8 + 2 * ARITH) * a * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)).all(), (causal, i)


def test_no_keys_and_empty(cuda):
    q = torch.ones(2, 3, 5, 64, dtype=torch.bfloat16, device=cuda)
    none = torch.ones(2, 3, 0, 64, dtype=torch.bfloat16, device=cuda)
    assert (sdk.sd_attention_masked(q, none, none) == 0).all()
    odd = torch.ones(2, 0, 3, 61, dtype=torch.bfloat16, device=cuda).transpose(1, 2)[..., :56]  # strides that no tensor map takes
    assert (sdk.sd_attention_masked(q[..., :56], odd, odd) == 0).all()
    assert (sdk.sd_attention_masked(q, none, none, causal=True, cap=3.0, bias=_bias(3, 4, 1, cuda)) == 0).all()
    assert sdk.sd_attention_masked(q[:, :, :0], q, q).shape == (2, 3, 0, 64)
    assert sdk.sd_attention_masked(q[:0], q[:0], q[:0]).shape == (0, 3, 5, 64)


def test_scale_zero_is_the_mean(cuda):
    q, k, v = _tensors(1, 2, 2, 140, 200, 64, torch.bfloat16, 91, cuda)
    _check(sdk.sd_attention_masked(q, k, v, scale=0.0, causal=True), q, k, v, scale=0.0, causal=True)


def test_two_captured_graphs_and_streams_at_once(cuda):
    # calls share no workspace: two graphs of split calls replayed together, on streams of their own
    q, k, v = _tensors(2, 8, 2, 1, 4000, 128, torch.bfloat16, 95, cuda, True)
    q2, k2, v2 = _tensors(2, 8, 2, 1, 4000, 128, torch.bfloat16, 96, cuda, True)
    want = [sdk.sd_attention_masked(*x, layout="blhd", causal=True) for x in ((q, k, v), (q2, k2, v2))]
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    for s, x in zip(streams, ((q, k, v), (q2, k2, v2))):
        s.wait_stream(torch.cuda.current_stream())
        o = torch.empty_like(x[0])
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                for _ in range(20):
                    sdk.sd_attention_masked(*x, layout="blhd", causal=True, out=o)
        graphs.append(g)
        outs.append(o)
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    sdk.sd_device_status()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_overlap_is_refused(cuda):
    big = torch.zeros(3, 2, 128, 64, dtype=torch.bfloat16, device=cuda)
    with pytest.raises(sdk.SDError, match="overlaps"):
        sdk.sd_attention_masked(big[:2], big[:2], big[:2], out=big[1:])
    with pytest.raises(sdk.SDError, match="heads overlap"):
        sdk.sd_attention_masked(big[:2], big[:2], big[:2], out=torch.zeros(4, 1, 128, 64, dtype=torch.bfloat16, device=cuda).as_strided((2, 2, 128, 64), (8192, 64, 64, 1)))


def test_few_queries_of_documents_split_over_a_cluster(cuda):
    # queries of three documents (one of them with no key) in one tile, against long keys
    q, k, v = _tensors(1, 4, 2, 90, 3000, 64, torch.bfloat16, 97, cuda, True)
    off = dict(q_offsets=_ints([2, 30, 31, 80], cuda), k_offsets=_ints([0, 1100, 1100, 2990], cuda))
    for kw in (dict(), dict(causal=True), dict(causal=True, q_starts=_ints([500, 0, -20], cuda)), dict(bias=_bias(4, 60, 98, cuda), cap=9.0)):
        out = torch.full_like(q, 7.0)
        kw = dict(kw, **off)
        o = sdk.sd_attention_masked(q, k, v, layout="blhd", out=out, **kw)
        _check(o, q, k, v, "blhd", out=torch.full_like(q, 7.0), **kw)


@pytest.mark.parametrize("cap", [1e-6, 0.3, 1e30])
def test_extreme_caps(cuda, cap):
    q, k, v = _tensors(1, 2, 2, 150, 200, 64, torch.bfloat16, 99, cuda)
    q[:, :, 5] = 0  # scores of exactly zero
    _check(sdk.sd_attention_masked(q, k, v, cap=cap), q, k, v, cap=cap)
    with pytest.raises(sdk.SDError, match="cap"):
        sdk.sd_attention_masked(q, k, v, scale=1.0, cap=1e-7)
    with pytest.raises(sdk.SDError, match="cap"):
        sdk.sd_attention_masked(q, k, v, scale=1e30, cap=1.0)
