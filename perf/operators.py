"""Measured cases of the transformer-block operators beside the UNet kernels.

Three operators make up a transformer block's path around its projections:

* ``rms``:    RMS norm with the residual's addition, with an output of the input's type or e4m3 with scales;
* ``rope``:   per-head RMS norm of q and k and rotary positions with several axes, in one pass;
* ``attend``: attention with causal, prefix, length and document masks, a tanh cap and a distance bias.

``run`` computes a case in elementary torch operations, or through the library where ``own`` is true.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the smallest scale: a block of zeros has it
GOLDEN = 0.6180339887498949


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # two tokens of a guided pair (unconditional, conditional) in a decoding step: launch latency
        {"name": "rms_token", "op": "rms", "rows": 2, "C": 1280, "dtype": "bf16", "residual": True, "fp8": False, "block": 0},
        # the 64 x 64 latent's tokens of a guided pair, normed into the 8-bit input of a projection
        {"name": "rms_latent_fp8", "op": "rms", "rows": 8192, "C": 1280, "dtype": "bf16", "residual": True, "fp8": True, "block": 128},
        # a video latent's tokens (21 x 30 x 52)
        {"name": "rms_video", "op": "rms", "rows": 32760, "C": 2048, "dtype": "bf16", "residual": True, "fp8": False, "block": 0},
        # an odd width in fp32, one scale a row: no vector of it is aligned
        {"name": "rms_odd_fp8", "op": "rms", "rows": 1001, "C": 1283, "dtype": "fp32", "residual": False, "fp8": True, "block": 0},
        # one new token of each of two sequences, heads shared by four queries: launch latency
        {"name": "rope_token", "op": "rope", "B": 2, "L": 1, "H": 16, "KV": 4, "dh": 128, "axes": "128", "dtype": "bf16", "pairs": "half",
         "norm": True, "fused": True, "far": 100000},
        # 77 text tokens and the 64 x 64 latent, read in place out of a fused projection's rows
        {"name": "rope_image", "op": "rope", "B": 2, "L": 4173, "H": 16, "KV": 16, "dh": 64, "axes": "16,24,24", "dtype": "bf16", "pairs": "interleaved",
         "norm": True, "fused": True, "far": 64},
        # a video latent, time x height x width
        {"name": "rope_video", "op": "rope", "B": 1, "L": 32760, "H": 16, "KV": 16, "dh": 128, "axes": "44,42,42", "dtype": "bf16", "pairs": "interleaved",
         "norm": True, "fused": False, "far": 64},
        # a pair of padded 77-token prompts in a causal text encoder
        {"name": "attend_prompt", "op": "attend", "B": 2, "H": 12, "KV": 12, "Lq": 77, "Lk": 77, "dh": 64, "dtype": "bf16", "layout": "blhd",
         "causal": True, "prefix": 0, "cap": 0.0, "radius": 0, "lens": True, "docs": 0},
        # padded 512-token prompts in an encoder whose scores get a learned bias by distance
        {"name": "attend_bias", "op": "attend", "B": 8, "H": 16, "KV": 16, "Lq": 512, "Lk": 512, "dh": 64, "dtype": "bf16", "layout": "blhd",
         "causal": False, "prefix": 0, "cap": 0.0, "radius": 128, "lens": True, "docs": 0},
        # images of several sizes with their prompts, packed in one sequence that is padded at its end
        {"name": "attend_packed", "op": "attend", "B": 1, "H": 10, "KV": 10, "Lq": 12288, "Lk": 12288, "dh": 64, "dtype": "bf16", "layout": "blhd",
         "causal": False, "prefix": 0, "cap": 0.0, "radius": 0, "lens": False, "docs": 7},
        # prompts that see themselves whole, then image tokens in raster order, with capped scores
        {"name": "attend_prefix_cap", "op": "attend", "B": 2, "H": 8, "KV": 8, "Lq": 4173, "Lk": 4173, "dh": 80, "dtype": "fp16", "layout": "bhld",
         "causal": True, "prefix": 77, "cap": 30.0, "radius": 0, "lens": False, "docs": 0},
        # one new token of each of 16 sequences against their caches, four queries to a key head
        {"name": "attend_decode", "op": "attend", "B": 16, "H": 16, "KV": 4, "Lq": 1, "Lk": 8192, "dh": 128, "dtype": "bf16", "layout": "blhd",
         "causal": True, "prefix": 0, "cap": 0.0, "radius": 0, "lens": True, "docs": 0},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rms", "rope", "attend", "attend"])
    if op == "rms":
        C = rng.choice([_spread(rng, 32, 8192), 8 * _spread(rng, 4, 1024), 320, 640, 1280, 2048])
        fp8 = rng.random() < 0.5
        return {"op": "rms", "rows": _spread(rng, 1, max(1, min(65536, (32760 * 2048) // C))), "C": C, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "residual": rng.random() < 0.6, "fp8": fp8, "block": rng.choice([0, 32, 64, 128]) if fp8 else 0}
    if op == "rope":
        dh, axes = rng.choice([(40, "8,16,16"), (64, "64"), (64, "16,24,24"), (64, "32,32"), (80, "40,40"), (80, "16,32,32"), (128, "44,42,42"), (128, "128"),
                               (128, "16,56,56"), (128, "32,32"), (160, "32,64,64")])
        B = rng.choice([1, 1, 2, 4])
        KV = rng.choice([1, 2, 4, 5, 8, 10])
        H = KV * rng.choice([1, 1, 2, 4])
        L = _spread(rng, 1, max(1, (32760 * 16 * 128) // (B * H * dh)))
        return {"op": "rope", "B": B, "L": L, "H": H, "KV": KV, "dh": dh, "axes": axes, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "pairs": rng.choice(["interleaved", "half"]), "norm": rng.random() < 0.6, "fused": rng.random() < 0.5, "far": rng.choice([64, 4096, 1000000])}
    dh = rng.choice([40, 64, 64, 80, 128, 128, 160])
    KV = rng.choice([1, 2, 4, 5, 8])
    H = KV * rng.choice([1, 1, 2, 4])
    form = rng.choice(["token", "encode", "encode", "packed"])
    causal = rng.random() < 0.5
    case = {"op": "attend", "H": H, "KV": KV, "dh": dh, "dtype": rng.choice(["bf16", "bf16", "fp16"]), "layout": rng.choice(["blhd", "bhld"]), "causal": causal,
            "cap": rng.choice([0.0, 0.0, 30.0, 50.0]), "radius": rng.choice([0, 0, 16, 128, 1000]), "prefix": 0, "lens": False, "docs": 0}
    if form == "token":
        case["B"] = _spread(rng, 1, 32)
        case["Lq"] = rng.choice([1, 1, 1, 2, 4, 7])
        case["Lk"] = max(case["Lq"], _spread(rng, 16, max(16, min(65536, (16 * 4 * 8192 * 128) // (case["B"] * KV * dh)))))
        case["lens"] = case["B"] > 1
    elif form == "encode":
        case["B"] = _spread(rng, 1, 8)
        most = max(64, math.isqrt(10 * 12288 * 4096 // (case["B"] * H)))
        case["Lk"] = _spread(rng, 33, min(6000, most))
        case["Lq"] = case["Lk"] if rng.random() < 0.7 else _spread(rng, 16, case["Lk"])
        case["lens"] = rng.random() < 0.5
        case["prefix"] = rng.choice([0, 77]) if causal else 0
    else:
        case["B"] = 1
        case["docs"] = _spread(rng, 1, 40)
        case["Lq"] = case["Lk"] = _spread(rng, 500, min(12288, math.isqrt(10 * 12288 * 12288 // H)))
    return {k: case[k] for k in ("op", "B", "H", "KV", "Lq", "Lk", "dh", "dtype", "layout", "causal", "prefix", "cap", "radius", "lens", "docs")}


# ------------------------------------------------------------------------------------------------ inputs
def _lens(case):
    """Key lengths of the batch, without their order: from a few keys to all of Lk."""
    lo = max(1, case["Lk"] // 8) if case["Lq"] == case["Lk"] else max(case["Lq"], case["Lk"] // 8)
    return [case["Lk"] if b == 0 else lo + int((case["Lk"] - lo) * ((GOLDEN * b) % 1.0)) for b in range(case["B"])]


def _docs(case):
    """Document lengths, without their order: together they leave about one row in 64 unused."""
    total, n = case["Lk"] - case["Lk"] // 64, case["docs"]
    share = [0.25 + (GOLDEN * (d + 1)) % 1.0 for d in range(n)]
    got = [max(1, int(total * s / sum(share))) for s in share]
    return got


def _generator(seed):
    return torch.Generator("cuda").manual_seed(int(seed))


def _order(n, seed):
    return np.random.RandomState(int(seed) % (1 << 32)).permutation(n)


def _frequencies(axes, theta=10000.0):
    """Turns a position, in units of 2^-64: theta^(-2 m / d) / (2 pi) for the pairs m of each axis of d columns."""
    f = [theta ** (-2.0 * m / d) / (2.0 * math.pi) for d in axes for m in range(d // 2)]
    return torch.tensor([int(round(x * 2.0 ** 64)) for x in f], dtype=torch.int64)


def _axes(case):
    return [int(d) for d in case["axes"].split(",")]


def prepare(case, seed):
    g = _generator(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "rms":
        rows, C = case["rows"], case["C"]
        s = {"case": case, "x": normal(rows, C).to(dt), "w": (1.0 + 0.1 * normal(C)).to(dt), "eps": 1e-6, "residual": None}
        if case["residual"]:
            s["residual"] = (4.0 * normal(rows, C)).to(dt)
        return s
    if case["op"] == "rope":
        B, L, H, KV, dh, axes = case["B"], case["L"], case["H"], case["KV"], case["dh"], _axes(case)
        if case["fused"]:  # views of a fused projection's rows [q heads | k heads | v heads]
            rows = normal(B, L, H + 2 * KV, dh).to(dt)
            q, k = rows[:, :, :H], rows[:, :, H:H + KV]
        else:
            q, k = normal(B, L, H, dh).to(dt), normal(B, L, KV, dh).to(dt)
        pos = torch.randint(0, case["far"], (B, L, len(axes)), generator=g, device="cuda", dtype=torch.int32)
        s = {"case": case, "q": q, "k": k, "positions": pos, "axes": axes, "freqs": _frequencies(axes).cuda(), "qw": None, "kw": None, "eps": 1e-6}
        if case["norm"]:
            s["qw"], s["kw"] = 1.0 + 0.1 * normal(dh), 1.0 + 0.1 * normal(dh)
        return s
    B, H, KV, Lq, Lk, dh = (case[k] for k in ("B", "H", "KV", "Lq", "Lk", "dh"))
    blhd = case["layout"] == "blhd"

    def rows(heads, L, spread=1.0):
        return (spread * normal(*((B, L, heads, dh) if blhd else (B, heads, L, dh)))).to(dt)

    s = {"case": case, "q": rows(H, Lq, 1.5), "k": rows(KV, Lk), "v": rows(KV, Lk), "scale": 1.0 / math.sqrt(dh), "bias": None,
         "kv_lens": None, "q_starts": None, "prefix_lens": None, "offsets": None, "out": None}
    if case["radius"]:
        R = case["radius"]
        d = torch.arange(-R, R + 1, device="cuda").abs().float()
        s["bias"] = -0.5 * torch.log1p(d)[None, :] * (1.0 + torch.arange(H, device="cuda")[:, None] / H) + 0.2 * normal(H, 2 * R + 1)
    ints = lambda v: torch.tensor([int(x) for x in v], dtype=torch.int32, device="cuda")  # noqa: E731
    if case["lens"]:
        lens = [_lens(case)[i] for i in _order(B, seed)]
        s["kv_lens"] = ints(lens)
        if Lq < Lk:  # the queries are the last rows of each sequence
            s["q_starts"] = ints([n - Lq for n in lens])
    if case["prefix"]:
        s["prefix_lens"] = ints([case["prefix"]] * B)
    if case["docs"]:
        lens = [_docs(case)[i] for i in _order(case["docs"], seed)]
        s["offsets"] = ints(np.cumsum([0] + lens))
        s["out"] = torch.zeros_like(s["q"])  # rows behind the last document stay as they are
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    return {"rms": _rms, "rope": _rope, "attend": _attend}[op](s)


def _own(s):
    import unet_latent_attention_b200 as sdk
    c = s["case"]
    if c["op"] == "rms":
        if not c["fp8"]:
            y = sdk.sd_rms_norm(s["x"], s["w"], s["eps"], residual=s["residual"])
            return dict(zip(("y", "residual"), y)) if c["residual"] else {"y": y}
        y = sdk.sd_rms_norm_fp8(s["x"], s["w"], s["eps"], residual=s["residual"], block=c["block"])
        return dict(zip(("y", "scales", "residual"), y))
    if c["op"] == "rope":
        q, k = sdk.sd_rope_axes(s["q"], s["k"], s["positions"], s["freqs"], s["axes"], pairs=c["pairs"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"])
        return {"q": q, "k": k}
    return {"o": sdk.sd_attention_masked(s["q"], s["k"], s["v"], scale=s["scale"], layout=c["layout"], causal=c["causal"], cap=c["cap"], bias=s["bias"],
                                         kv_lens=s["kv_lens"], q_starts=s["q_starts"], prefix_lens=s["prefix_lens"], q_offsets=s["offsets"],
                                         k_offsets=s["offsets"], out=s["out"])}


def _rms(s):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * w; in e4m3, each block of a row over its largest magnitude / 448."""
    c = s["case"]
    h = s["x"].float()
    if c["residual"]:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"]) * s["w"].float()
    got = {}
    if c["fp8"]:
        rows, C = y.shape
        block = c["block"] or C
        n = -(-C // block)
        t = torch.nn.functional.pad(y, (0, n * block - C)).view(rows, n, block)
        scales = (t.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
        got["y"] = (t / scales[..., None]).view(rows, n * block)[:, :C].to(torch.float8_e4m3fn)
        got["scales"] = scales
    else:
        got["y"] = y.to(s["x"].dtype)
    if c["residual"]:
        got["residual"] = h.to(s["x"].dtype)
    return got


def _rotate(x, cos, sin, half):
    """Turns the pairs of the first 2 * cos.shape[-1] columns of x [B, L, heads, dh] by angles [B, L, 1, pairs]."""
    n = cos.shape[-1]
    a, b = (x[..., :n], x[..., n:2 * n]) if half else (x[..., 0:2 * n:2], x[..., 1:2 * n:2])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat((u, v), -1) if half else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((turned, x[..., 2 * n:]), -1)


def _rope(s):
    axis = torch.repeat_interleave(torch.arange(len(s["axes"]), device="cuda"), torch.tensor([d // 2 for d in s["axes"]], device="cuda"))
    turns = s["positions"].double()[..., axis] * (s["freqs"].double() * 2.0 ** -64)  # far positions: the angle in 64 bits
    angle = (2.0 * math.pi * (turns - turns.round()))[:, :, None]
    cos, sin = angle.cos().float(), angle.sin().float()

    def one(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w
        return _rotate(y, cos, sin, s["case"]["pairs"] == "half").to(x.dtype)

    return {"q": one(s["q"], s["qw"]), "k": one(s["k"], s["kw"])}


def _heads_first(s, t):
    return t.transpose(1, 2) if s["case"]["layout"] == "blhd" else t


def _visible(s):
    """(which keys each query sees [S, Lq, Lk], key position - query position [S, Lq, Lk]); S is the batch, or 1."""
    c = s["case"]
    i = torch.arange(c["Lq"], device="cuda")[None, :, None]
    j = torch.arange(c["Lk"], device="cuda")[None, None, :]
    if s["offsets"] is not None:
        off = s["offsets"].long()
        qd, kd = torch.searchsorted(off, i, right=True), torch.searchsorted(off, j, right=True)
        see = (qd == kd) & (qd <= c["docs"])
        dist = j - i  # each document has as many queries as keys
        return see & (dist <= 0) if c["causal"] else see, dist
    start = s["q_starts"].long()[:, None, None] if s["q_starts"] is not None else c["Lk"] - c["Lq"]
    dist = j - (i + start)
    see = j < (s["kv_lens"].long()[:, None, None] if s["kv_lens"] is not None else c["Lk"])
    if c["causal"]:
        seen = dist <= 0
        if s["prefix_lens"] is not None:
            seen = seen | (j < s["prefix_lens"].long()[:, None, None])
        see = see & seen
    return see.expand(-1, c["Lq"], -1), dist


def _attend(s):
    c = s["case"]
    B, H, KV, Lq, Lk, dh = (c[k] for k in ("B", "H", "KV", "Lq", "Lk", "dh"))
    G = H // KV
    q, k, v = (_heads_first(s, s[n]).float() for n in ("q", "k", "v"))
    t = torch.matmul(q.reshape(B, KV, G * Lq, dh), k.transpose(-1, -2)).view(B, KV, G, Lq, Lk) * s["scale"]
    if c["cap"]:
        t = c["cap"] * torch.tanh(t / c["cap"])
    see, dist = _visible(s)
    if s["bias"] is not None:
        R = c["radius"]
        t = t + s["bias"][:, (dist.clamp(-R, R) + R)].transpose(0, 1).reshape(-1, KV, G, Lq, Lk)
    t = t.masked_fill(~see[:, None, None], -math.inf)
    top = t.amax(-1, keepdim=True)
    p = torch.exp(t - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, KV, G * Lq, Lk), v).view(B, H, Lq, dh) / torch.where(total == 0, 1.0, total).view(B, H, Lq, 1)
    o = o.to(s["q"].dtype)
    if c["layout"] == "blhd":
        o = o.transpose(1, 2)
    if s["out"] is not None:
        inside = (torch.arange(Lq, device="cuda") < s["offsets"][-1]).view((1, Lq, 1, 1) if c["layout"] == "blhd" else (1, 1, Lq, 1))
        return {"o": torch.where(inside, o, s["out"])}
    return {"o": o.contiguous()}


# ------------------------------------------------------------------------------------------------ work
def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if case["op"] == "rms":
        rows, C, n = case["rows"], case["C"], 1 + (2 if case["residual"] else 0)  # x, and the residual in and out
        out = rows * C + rows * 4 * (-(-C // case["block"]) if case["block"] else 1) if case["fp8"] else rows * C * size
        return {"bytes": rows * C * size * n + out + C * size, "flops": 4 * rows * C}
    if case["op"] == "rope":
        n = case["B"] * case["L"] * (case["H"] + case["KV"]) * case["dh"]
        return {"bytes": 2 * n * size + 4 * case["B"] * case["L"] * len(_axes(case)), "flops": 3 * n + (4 * n if case["norm"] else 0)}
    B, H, KV, Lq, Lk, dh = (case[k] for k in ("B", "H", "KV", "Lq", "Lk", "dh"))
    if case["docs"]:
        sets = [(n, n, 0) for n in _docs(case)]
    else:
        lens = _lens(case) if case["lens"] else [Lk] * B
        sets = [(Lq, n, (n - Lq) if case["lens"] and Lq < Lk else Lk - Lq) for n in lens]
    pairs = q_rows = k_rows = 0
    for nq, nk, start in sets:
        q_rows, k_rows = q_rows + nq, k_rows + nk
        if case["causal"]:
            i = np.arange(nq, dtype=np.int64)
            pairs += int(np.clip(np.maximum(start + i + 1, case["prefix"]), 0, nk).sum())
        else:
            pairs += nq * nk
    return {"bytes": size * dh * (2 * q_rows * H + 2 * k_rows * KV), "flops": 4 * pairs * H * dh}


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rms": _exact_rms, "rope": _exact_rope, "attend": _exact_attend}[case["op"]](s)


def _exact_rms(s):
    c = s["case"]
    h = s["x"].double() + (s["residual"].double() if c["residual"] else 0.0)
    C = h.shape[1]
    y = h / (torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / C + s["eps"]).sqrt() * s["w"].double()
    got = {"residual": h} if c["residual"] else {}
    if not c["fp8"]:
        return {"y": y, **got}
    edges = list(range(0, C, c["block"] or C))
    scales = torch.stack([y[:, e:e + (c["block"] or C)].abs().max(1).values.div(448).clamp_min(TINY) for e in edges], 1)
    of = torch.arange(C, device="cuda") // (c["block"] or C)
    return {"y": y / scales[:, of], "scales": scales, **got}


def _exact_rope(s):
    c = s["case"]
    half = sum(s["axes"]) // 2

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["dh"] + s["eps"]).sqrt() * w.double()
        y, m = x.clone(), 0
        for a, d in enumerate(s["axes"]):
            for r in range(d // 2):
                f = 10000.0 ** (-2.0 * r / d)
                z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), (s["positions"][..., a].double() * f))[:, :, None]
                i, j = (m, m + half) if c["pairs"] == "half" else (2 * m, 2 * m + 1)
                turned = torch.complex(x[..., i], x[..., j]) * z
                y[..., i], y[..., j] = turned.real, turned.imag
                m += 1
        return y

    return {"q": one(s["q"], s["qw"]), "k": one(s["k"], s["kw"])}


def _exact_attend(s):
    c = s["case"]
    B, H, KV, Lq, Lk = (c[k] for k in ("B", "H", "KV", "Lq", "Lk"))
    q, k, v = (_heads_first(s, s[n]).double() for n in ("q", "k", "v"))
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    if s["offsets"] is not None:
        off = s["offsets"].tolist()
        parts = [(0, a, b, a, b, 0, 0) for a, b in zip(off, off[1:])]
    else:
        lens = s["kv_lens"].tolist() if s["kv_lens"] is not None else [Lk] * B
        starts = s["q_starts"].tolist() if s["q_starts"] is not None else [Lk - Lq] * B
        parts = [(b, 0, Lq, 0, lens[b], starts[b], c["prefix"]) for b in range(B)]
    for b, q0, q1, k0, k1, start, prefix in parts:
        if k1 <= k0 or q1 <= q0:
            continue
        at = start + torch.arange(q1 - q0, device="cuda")[:, None]
        key = torch.arange(k1 - k0, device="cuda")[None, :]
        hidden = (key > at) & (key >= prefix) if c["causal"] else None
        for h in range(H):
            t = q[b, h, q0:q1] @ k[b, h * KV // H, k0:k1].T * s["scale"]
            if c["cap"]:
                t = torch.tanh(t / c["cap"]) * c["cap"]
            if s["bias"] is not None:
                R = c["radius"]
                t += s["bias"][h].double()[torch.clamp(key - at, -R, R) + R]
            if hidden is not None:
                t[hidden] = -math.inf
            w = torch.softmax(t, 1).nan_to_num(0.0) if hidden is not None else torch.softmax(t, 1)
            o[b, h, q0:q1] = w @ v[b, h * KV // H, k0:k1]
    return {"o": o.transpose(1, 2) if c["layout"] == "blhd" else o}
