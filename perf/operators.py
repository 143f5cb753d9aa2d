"""Cases and plain forms of the transformer-block operators that stand between the quantized
linears: the residual's addition with root-mean-square norm and an 8-bit output, the matrix
product with bias, activation and residual in its epilogue, and the rotary positions with
several axes.

Each case is one call of one operator.  run() computes it in elementary fp32 torch operations
(own = False) or through the framework's binding (own = True), on the same inputs.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
          "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "int8": 1, "e4m3": 1, "same": 2}
QMAX = {"int8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -100          # floor of a row's absolute maximum: a row of zeros gets codes 0 and a finite scale
EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------ cases
def _norm(name, M, K, x="bf16", residual="same", out="int8", weight="f32", pad=0):
    return {"op": "norm", "name": name, "M": M, "K": K, "x": x, "residual": residual, "out": out,
            "weight": weight, "pad": pad}


def _gemm(name, M, K, N, types="int8", out="bf16", act="none", bias=True, residual=False):
    return {"op": "gemm", "name": name, "M": M, "K": K, "N": N, "types": types, "out": out, "act": act,
            "bias": bias, "residual": residual}


def _rope(name, batch, tokens, heads, kv_heads, dim, axes, pairs="adjacent", dtype="f16", norm=True,
          heads_first=False, inverse=False, text=0, width=64):
    """axes: pairs of each axis, e.g. "8,28,28" (time, height, width)."""
    return {"op": "rope", "name": name, "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "axes": axes, "pairs": pairs, "dtype": dtype, "norm": norm, "heads_first": heads_first,
            "inverse": inverse, "text": text, "width": width}


def listed():
    return [
        # one token's residual stream before a block's 8-bit linear: latency alone
        _norm("norm 1x3072", 1, 3072, x="bf16", out="int8"),
        # a 4608-token sequence (4096 image + 512 text tokens), 16-bit stream, FP8 codes
        _norm("norm 4608x3072 e4m3", 4608, 3072, x="f16", out="e4m3"),
        # four such sequences with the stream held in 32 bits
        _norm("norm 18432x3072 f32 stream", 18432, 3072, x="bf16", residual="f32", out="int8"),
        # odd width and a padded row stride, no residual, 16-bit output (the input of a W4A4 layer)
        _norm("norm 777x1111 strided", 777, 1111, x="f16", residual="none", out="same", weight="f16", pad=3),
        # one token through an MLP's first 8-bit linear: the weight's bytes bound it
        _gemm("gemm int8 1x3072x12288 gelu", 1, 3072, 12288, types="int8", out="f16", act="gelu"),
        # 64 tokens through the MLP's second linear and onto the residual stream
        _gemm("gemm e4m3 64x12288x3072 res", 64, 12288, 3072, types="e4m3", out="bf16", residual=True),
        # an MLP's first linear at 4608 tokens: the largest product
        _gemm("gemm int8 4608x3072x12288 gelu", 4608, 3072, 12288, types="int8", out="f16", act="gelu"),
        # 512 text tokens through a projection kept at 16 bits
        _gemm("gemm bf16 512x3072x9216", 512, 3072, 9216, types="bf16", out="bf16"),
        # ragged sizes that end inside every tile
        _gemm("gemm f16 333x1048x1999 silu res", 333, 1048, 1999, types="f16", out="f16", act="silu", residual=True),
        # one decoded token, 24 heads of 128, both norms: latency alone
        _rope("rope 1 token 24 heads", 1, 1, 24, 24, 128, "8,28,28"),
        # queries and keys of a packed projection, 512 text tokens then a 64 x 64 image, both norms
        _rope("rope 4608 tokens 3 axes", 1, 4608, 24, 24, 128, "8,28,28", text=512),
        # two videos (time, height, width), shared key heads, half-apart pairs, head-major output
        _rope("rope 2x16384 video shared", 2, 16384, 32, 8, 128, "16,24,24", pairs="halves", dtype="bf16", norm=False,
              heads_first=True, width=52),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gemm", "rope"])
    if op == "norm":
        K = _log(rng, 16, 12288)
        if rng.random() < 0.6:
            K = -(-K // 16) * 16
        M = _log(rng, 1, max(1, min(18432, 18432 * 3072 // K)))
        c = _norm("", M, K, x=rng.choice(["f16", "bf16"]), residual=rng.choice(["same", "f32", "none"]),
                  out=rng.choice(["int8", "e4m3", "same"]), weight=rng.choice(["f32", "x"]), pad=rng.choice([0, 0, 8, 5]))
        c["weight"] = c["x"] if c["weight"] == "x" else "f32"
    elif op == "gemm":
        types = rng.choice(["int8", "e4m3", "f16", "bf16"])
        K = _log(rng, 64, 12288) // 16 * 16
        N = _log(rng, 16, 12288)
        if rng.random() < 0.6:
            N = -(-N // 16) * 16
        # the time of a 16-bit product is twice an 8-bit one's
        most = 4608 * 3072 * 12288 // (K * N * (1 if types in ("int8", "e4m3") else 2))
        c = _gemm("", _log(rng, 1, max(1, min(4608, most))), K, N, types=types, out=rng.choice(["f16", "bf16"]),
                  act=rng.choice(["none", "gelu", "silu"]), bias=rng.random() < 0.7, residual=rng.random() < 0.5)
    else:
        dim = rng.choice([64, 72, 80, 96, 128, 128, 256])
        axes = rng.choice([1, 2, 3, 3])
        half = dim // 2 if rng.random() < 0.7 else dim // 4
        cut = sorted(rng.sample(range(1, half), axes - 1))
        parts = [b - a for a, b in zip([0] + cut, cut + [half])]
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4])
        batch = rng.choice([1, 1, 2, 3])
        most = 2 * 16384 * 40 * 128 // (batch * (heads + kv) * dim)
        c = _rope("", batch, _log(rng, 1, min(32768, most)), heads, kv, dim, ",".join(map(str, parts)),
                  pairs=rng.choice(["adjacent", "halves"]), dtype=rng.choice(["f16", "bf16"]), norm=rng.random() < 0.5,
                  heads_first=rng.random() < 0.5, text=rng.choice([0, 0, 77]), width=rng.choice([13, 32, 64]))
        c["inverse"] = not c["norm"] and rng.random() < 0.3
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _outliers(g, x):
    """1% of the channels 30 times larger, as activations of these layers have."""
    K = x.shape[-1]
    scale = torch.ones(K, device="cuda")
    scale[torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]] = 30.0
    return x * scale


def _quantized(v, types):
    """Codes of v's rows and their fp32 scales."""
    a = v.abs().amax(-1, keepdim=True).clamp_min(TINY)
    c = v * (torch.full_like(a, QMAX[types]) / a)
    c = c.round().to(torch.int8) if types == "int8" else c.to(torch.float8_e4m3fn)
    return c, (a / QMAX[types]).squeeze(-1).contiguous()


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "norm":
        M, K, pad = c["M"], c["K"], c["pad"]
        x, r = DTYPES[c["x"]], DTYPES[c["x"] if c["residual"] == "same" else "f32"]
        s["x"] = _randn(g, M, K + pad).to(x)[:, :K]
        s["residual"] = None if c["residual"] == "none" else _outliers(g, _randn(g, M, K)).to(r)
        s["weight"] = (1.0 + 0.1 * _randn(g, K)).to(DTYPES[c["weight"]])
    elif c["op"] == "gemm":
        M, K, N, out = c["M"], c["K"], c["N"], DTYPES[c["out"]]
        x, w = _outliers(g, _randn(g, M, K)), _randn(g, N, K) / math.sqrt(K)
        if c["types"] in QMAX:
            s["x"], s["xs"] = _quantized(x, c["types"])
            s["w"], s["ws"] = _quantized(w, c["types"])
        else:
            s["x"], s["w"], s["xs"], s["ws"] = x.to(DTYPES[c["types"]]), w.to(DTYPES[c["types"]]), None, None
        s["bias"] = _randn(g, N).to(out) if c["bias"] else None
        s["residual"] = _randn(g, M, N).to(out) if c["residual"] else None
    else:
        B, T, H, G, D, dt = c["batch"], c["tokens"], c["heads"], c["kv_heads"], c["dim"], DTYPES[c["dtype"]]
        s["axes"] = tuple(int(a) for a in c["axes"].split(","))
        qkv = _randn(g, B, T, (H + 2 * G) * D).to(dt)      # a packed projection, read in place
        s["q"] = qkv[..., : H * D].unflatten(-1, (H, D))
        s["k"] = qkv[..., H * D:(H + G) * D].unflatten(-1, (G, D))
        # positions (time, height, width) of a grid behind `text` tokens at the origin, from a frame the seed picks
        i = (torch.arange(T, device="cuda") - c["text"]).clamp_min(0)
        first = int(torch.randint(0, 1000, (1,), generator=g, device="cuda"))
        W = c["width"]
        grid = [first + i // (W * W), i // W % W, i % W] if len(s["axes"]) == 3 else [first + i // W, i % W]
        grid = [first + i] if len(s["axes"]) == 1 else grid
        s["positions"] = torch.stack(grid, -1).to(torch.int32)
        s["inv_freq"] = torch.cat([THETA ** (-torch.arange(n, device="cuda", dtype=torch.float64) / n)
                                   for n in s["axes"]]).float()
        s["axis"] = torch.cat([torch.full((n,), a, device="cuda") for a, n in enumerate(s["axes"])])   # of each pair
        s["qw"] = (1.0 + 0.1 * _randn(g, D)) if c["norm"] else None
        s["kw"] = (1.0 + 0.1 * _randn(g, D)) if c["norm"] else None
        # attention's layout: token-major, or head-major [batch, heads, tokens, dim]
        s["heads_first"] = c["heads_first"]
    return s


# ------------------------------------------------------------------ one pass
def _plain_norm(s, c):
    h = s["x"].float()
    stream = None
    if s["residual"] is not None:
        stream = (h + s["residual"].float()).to(s["residual"].dtype)
        h = stream.float()
    rstd = 1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS)
    v = h * s["weight"].float()
    if c["out"] == "same":
        return {"out": (v * rstd).to(s["x"].dtype), "stream": stream}
    # the norm is a factor of the whole row, so the codes do not depend on it
    a = v.abs().amax(-1, keepdim=True).clamp_min(TINY)
    q = v * (torch.full_like(a, QMAX[c["out"]]) / a)
    q = q.round().to(torch.int8) if c["out"] == "int8" else q.to(torch.float8_e4m3fn)
    return {"out": q, "scales": (a * rstd / QMAX[c["out"]]).squeeze(-1), "stream": stream}


def _plain_gemm(s, c):
    y = s["x"].float() @ s["w"].float().t()
    if s["xs"] is not None:
        y = y * s["xs"][:, None] * s["ws"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    elif c["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[c["out"]])


def _turned(x, w, cos, sin, c):
    """One of queries or keys [batch, tokens, heads, dim]; cos, sin [tokens, 1, pairs]."""
    v = x.float()
    if w is not None:
        v = v * (1.0 / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)) * w
    P = cos.shape[-1]
    turned, rest = v[..., : 2 * P], v[..., 2 * P:]
    if c["pairs"] == "adjacent":
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = turned[..., :P], turned[..., P:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, rest), -1).to(x.dtype)


def _plain_rope(s, c):
    angle = s["positions"].float()[:, s["axis"]] * s["inv_freq"]
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    if c["inverse"]:
        sin = -sin
    out = {}
    for name, x, w in (("q", s["q"], s["qw"]), ("k", s["k"], s["kw"])):
        y = _turned(x, w, cos, sin, c)
        out[name] = y.transpose(1, 2).contiguous() if s["heads_first"] else y
    return out


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _plain_norm, "gemm": _plain_gemm, "rope": _plain_rope}[c["op"]](s, c)
    from bit_w4a4_quantized_amd import binding
    if c["op"] == "norm":
        out, scales, stream = binding.svdq_add_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"],
                                                       out_format=c["out"])
        return {"out": out, "stream": stream} if scales is None else {"out": out, "scales": scales, "stream": stream}
    if c["op"] == "gemm":
        return binding.svdq_gemm_act_residual(s["x"], s["w"], xs=s["xs"], ws=s["ws"], bias=s["bias"],
                                              activation=c["act"], residual=s["residual"], out_dtype=DTYPES[c["out"]])
    q, k = binding.svdq_rope_axes(s["q"], s["k"], s["positions"], s["inv_freq"], s["axes"], pairs=c["pairs"],
                                  q_weight=s["qw"], k_weight=s["kw"], eps=EPS, inverse=c["inverse"],
                                  heads_first=s["heads_first"])
    return {"q": q, "k": k}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "norm":
        n = c["M"] * c["K"]
        stream = {"same": 2, "f32": 4, "none": 0}[c["residual"]]
        return {"bytes": n * (2 + 2 * stream + SIZE[c["out"]]) + c["K"] * SIZE[c["weight"]] +
                (0 if c["out"] == "same" else 4 * c["M"]), "flops": 6 * n}
    if c["op"] == "gemm":
        M, K, N, b = c["M"], c["K"], c["N"], SIZE[c["types"]]
        return {"bytes": (M + N) * (K * b + (4 if b == 1 else 0)) + 2 * M * N * (2 if c["residual"] else 1) +
                (2 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    n = c["batch"] * c["tokens"] * (c["heads"] + c["kv_heads"]) * c["dim"]
    axes = c["axes"].count(",") + 1
    return {"bytes": 4 * n + 4 * c["tokens"] * axes, "flops": (7 if c["norm"] else 3) * n}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    d = lambda t: t.to(torch.float64)  # noqa: E731
    if c["op"] == "norm":
        h, out = d(s["x"]), {}
        if s["residual"] is not None:
            out["stream"] = h + d(s["residual"])
            h = d(out["stream"].to(s["residual"].dtype))    # the stream as it is kept
        else:
            out["stream"] = None
        root = (h.pow(2).sum(-1) / c["K"] + EPS).rsqrt()
        g = h * d(s["weight"])
        if c["out"] == "same":
            out["out"] = g * root[:, None]
        else:
            top = g.abs().max(-1).values.clamp_min(TINY)
            out["scales"] = top * root / QMAX[c["out"]]
            out["out"] = None if c["out"] == "int8" else g / top[:, None] * QMAX[c["out"]]
        return out
    if c["op"] == "gemm":
        z = torch.mm(d(s["x"]), d(s["w"]).T)
        if s["xs"] is not None:
            z = torch.outer(d(s["xs"]), d(s["ws"])) * z
        z = z if s["bias"] is None else z + d(s["bias"])
        if c["act"] == "gelu":      # 0.5 (1 + tanh u) = 1 / (1 + e^(-2u))
            z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3)))
        elif c["act"] == "silu":
            z = z * torch.sigmoid(z)
        return z if s["residual"] is None else z + d(s["residual"])
    # each pair as a complex number, multiplied by exp(i angle)
    at = sum(([i] * n for i, n in enumerate(s["axes"])), [])
    angle = d(s["positions"])[:, at] * d(s["inv_freq"])
    turn = torch.polar(torch.ones_like(angle), -angle if c["inverse"] else angle)[None, :, None]
    out = {}
    for name, x, w in (("q", d(s["q"]), s["qw"]), ("k", d(s["k"]), s["kw"])):
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + EPS).sqrt() * d(w)
        P, y = angle.shape[-1], x.clone()
        low = slice(0, 2 * P, 2) if c["pairs"] == "adjacent" else slice(0, P)
        high = slice(1, 2 * P, 2) if c["pairs"] == "adjacent" else slice(P, 2 * P)
        z = torch.complex(x[..., low], x[..., high]) * turn
        y[..., low], y[..., high] = z.real, z.imag
        out[name] = y.permute(0, 2, 1, 3).contiguous() if s["heads_first"] else y
    return out
