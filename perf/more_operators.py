"""Cases and plain forms of the operators around a paged cache of keys and values: appending a
step's tokens with their rotary positions, attention of drafted tokens (a tree, or a plain chain)
over the cache, and keeping the accepted path of a draft.

Each case is one call of one operator.  run() computes it in elementary fp32 torch operations
(own = False) or through the framework's binding (own = True), on the same inputs.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
SIZE = {"f16": 2, "bf16": 2, "int8": 1, "e4m3": 1}
QMAX = {"int8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -100          # floor of a head's absolute maximum: a head of zeros gets codes 0 and a finite scale
EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------ cases
def _case(op, name, sequences, tokens, context, heads, kv_heads, dim, dtype="bf16", cache="same", page=64, ragged=False,
          **more):
    """tokens: of each sequence in this step (at most, when ragged); context: of each in the cache before it."""
    return {"op": op, "name": name, "sequences": sequences, "tokens": tokens, "context": context, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "cache": dtype if cache == "same" else cache, "page": page,
            "ragged": ragged, **more}


def _append(*a, axes="", pairs="halves", norm=False, **kw):
    return _case("append", *a, axes=axes or str(a[6] // 2), pairs=pairs, norm=norm, **kw)


def _attention(*a, tree=True, **kw):
    return _case("attention", *a, tree=tree, **kw)


def _keep(*a, path=8, **kw):
    return _case("keep", *a, path=path, **kw)


def listed():
    return [
        # one decoded token into an FP8 cache: latency alone
        _append("append 1 token e4m3", 1, 1, 1000, 32, 8, 128, cache="e4m3", page=16),
        # 64 sequences decode a token each, 16-bit cache
        _append("append 64 x 1 bf16", 64, 1, 2000, 32, 8, 128),
        # drafted trees of a few sequences, heads of 80 in small pages
        _append("append 13 x 61 dim 80", 13, 61, 500, 10, 10, 80, dtype="f16", page=8, ragged=True, pairs="adjacent"),
        # four prompts of text and image, normed heads with three axes, into an FP8 cache
        _append("append 4 x 4096 e4m3", 4, 4096, 0, 24, 24, 128, dtype="f16", cache="e4m3", axes="8,28,28",
                pairs="adjacent", norm=True),
        # one sequence decodes one token over a short cache: latency alone
        _attention("decode 1 over 1000", 1, 1, 999, 32, 8, 128, page=16),
        # a serving batch decodes a token each over 8-bit caches of mixed lengths: the cache's bytes bound it
        _attention("decode 64 over 8000 int8", 64, 1, 8000, 32, 8, 128, cache="int8", ragged=True),
        # one sequence decodes over a long FP8 cache: split over its length
        _attention("decode 1 over 131071 e4m3", 1, 1, 131071, 32, 8, 128, dtype="f16", cache="e4m3"),
        # trees of 61 drafted tokens checked for 16 sequences
        _attention("tree 16 x 61 over 6000", 16, 61, 6000, 32, 8, 128, ragged=True),
        # small trees, heads of 80 without sharing, pages that end inside every tile
        _attention("tree 5 x 37 dim 80", 5, 37, 1777, 10, 10, 80, dtype="f16", page=8, ragged=True),
        # a chunk of a long prompt over what precedes it: the largest, the matrix cores bound it
        _attention("chunk 4096 over 12288", 1, 4096, 12288, 24, 24, 128, tree=False),
        # one sequence keeps five of 61 drafted tokens: latency alone
        _keep("keep 1 x 5", 1, 61, 1000, 32, 8, 128, page=16, path=5),
        # a serving batch keeps up to eight each
        _keep("keep 256 x 8 e4m3", 256, 61, 600, 32, 8, 128, cache="e4m3", ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "keep"])
    dim = rng.choice([64, 80, 96, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["f16", "bf16"])
    kw = dict(dtype=dtype, cache=rng.choice([dtype, dtype, "int8", "e4m3"]), page=rng.choice([8, 16, 32, 64, 128, 256]),
              ragged=rng.random() < 0.7)
    sequences = _log(rng, 1, 128)
    if op == "append":
        axes = rng.choice([1, 1, 2, 3])
        half = dim // 2 if rng.random() < 0.7 else dim // 4
        cut = sorted(rng.sample(range(1, half), axes - 1))
        parts = [b - a for a, b in zip([0] + cut, cut + [half])]
        tokens = _log(rng, 1, max(1, min(16384, 4 * 4096 * 72 * 128 // (sequences * (heads + 2 * kv) * dim))))
        c = _append("", sequences, tokens, _log(rng, 1, 1000), heads, kv, dim, axes=",".join(map(str, parts)),
                    pairs=rng.choice(["adjacent", "halves"]), norm=rng.random() < 0.4, **kw)
    elif op == "attention":
        tree = rng.random() < 0.7
        tokens = 1 if rng.random() < 0.3 else _log(rng, 2, 130) if tree else _log(rng, 2, 4096)
        # neither more products than the largest chunk's, nor more plain logits, nor more cache than a long one's
        most = 4096 * 14336 * 24 * 128 // (sequences * tokens * heads * dim)
        most = min(most, 64 * 8000 * 8 * 128 // (sequences * kv * dim), 4096 * 16384 * 24 // (sequences * tokens * heads))
        c = _attention("", sequences, tokens, _log(rng, 1, max(2, min(131072, most))), heads, kv, dim, tree=tree, **kw)
    else:
        path = rng.randint(1, 12)
        c = _keep("", sequences, path + rng.randint(1, 100), _log(rng, 1, max(2, min(4000, 256 * 600 * 8 * 128 // (sequences * kv * dim)))),
                  heads, kv, dim, path=path, **kw)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _quantized(v, types):
    """Codes of v's heads and their fp32 scales."""
    a = v.abs().amax(-1, keepdim=True).clamp_min(TINY)
    c = v * (torch.full_like(a, QMAX[types]) / a)
    c = c.round().to(torch.int8) if types == "int8" else c.to(torch.float8_e4m3fn)
    return c, (a / QMAX[types]).squeeze(-1)


def _spread(n, low, most, ragged, shift=0.0):
    """n whole numbers, `most` or spread evenly over low ... most in a mixed order: the case's, whatever the seed."""
    if not ragged:
        return torch.full((n,), most, device="cuda")
    place = (0.6180339887 * torch.arange(1, n + 1, device="cuda", dtype=torch.float64) + shift) % 1.0
    return low + (place * (most - low + 1)).long().clamp_max(most - low)


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    B, T, H, G, D, page = c["sequences"], c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    dt, types = DTYPES[c["dtype"]], c["cache"]
    s = {"case": c}
    # the step's tokens of each sequence behind one another, and what each has in the cache before them
    count = _spread(B, c["path"] + 1 if c["op"] == "keep" else max(1, T // 2), T, c["ragged"])
    s["context"] = _spread(B, c["context"] // 2, c["context"], c["ragged"], 0.5).int()
    s["starts"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).int()
    s["n"] = N = int(s["starts"][-1])
    # pages handed out in any order, some left over; -1 behind a sequence's last
    need = (s["context"] + count + page - 1) // page
    width = int(need.max())
    pages = B * width + 3
    ids = torch.randperm(pages, generator=g, device="cuda")[: B * width].view(B, width)
    s["table"] = torch.where(torch.arange(width, device="cuda") < need[:, None], ids, -1).int()
    # the sequence of each token, and its place there
    s["of"] = torch.repeat_interleave(torch.arange(B, device="cuda"), count, output_size=N)
    s["at"] = torch.arange(N, device="cuda") - s["starts"][s["of"]]
    for name in ("k", "v"):
        x = _randn(g, pages, page, G, D)
        x[..., : max(1, D // 64)] *= 4.0                   # a few channels far larger, as keys and values have
        s[name + "_scales"] = None
        if types in QMAX:
            s[name], s[name + "_scales"] = _quantized(x, types)
        else:
            s[name] = x.to(dt)
        del x
    if c["op"] == "append":
        s["axes"] = tuple(int(a) for a in c["axes"].split(","))
        qkv = _randn(g, N, (H + 2 * G) * D).to(dt)         # a packed projection, read in place
        s["new"] = [t.unflatten(-1, (-1, D)) for t in qkv.split([H * D, G * D, G * D], -1)]
        # positions: behind the context along the last axis, a 64 x 64 grid before it from a frame that the seed picks
        i = s["context"][s["of"]].long() + s["at"]
        first = int(torch.randint(0, 1000, (1,), generator=g, device="cuda"))
        grid = [[first + i], [first + i // 64, i % 64], [first + i // 4096, i // 64 % 64, i % 64]][len(s["axes"]) - 1]
        s["positions"] = torch.stack(grid, -1).int()
        s["inv_freq"] = torch.cat([THETA ** (-torch.arange(n, device="cuda", dtype=torch.float64) / n)
                                   for n in s["axes"]]).float()
        s["qw"], s["kw"] = (1.0 + 0.1 * _randn(g, D), 1.0 + 0.1 * _randn(g, D)) if c["norm"] else (None, None)
    elif c["op"] == "attention":
        s["q"] = (2.0 * _randn(g, N, H, D)).to(dt)
        s["tree"] = None
        if c["tree"]:
            # each token hangs from any before it and sees itself and its ancestors
            j = torch.arange(T, device="cuda")
            up = (_rand(g, B, T) * j).long()
            sees = torch.eye(T, device="cuda").expand(B, T, T).clone()
            sees.scatter_(2, up[:, :, None], 1.0)
            for _ in range(max(1, (T - 1).bit_length())):
                sees = (torch.bmm(sees, sees) > 0).float()
            s["tree"] = sees[s["of"], s["at"]] > 0
    else:
        # the first drafted token and others from behind the path's length, in order; -1 ends a path
        P = c["path"]
        key = _rand(g, B, T)
        key[torch.arange(T, device="cuda") >= count[:, None]] = 2.0
        key[:, :P] = 2.0
        kept = key.argsort(1)[:, : P].sort(1).values
        kept[:, 0] = 0
        have = torch.minimum(_spread(B, 1, P, B > 1, 0.25), (count - P + 1).clamp_min(1))
        order = torch.arange(P, device="cuda")
        kept = torch.where(key.gather(1, kept) < 2.0, kept, T)        # places that held none of the sequence's tokens
        kept[:, 0] = 0
        kept = kept.sort(1).values
        s["path"] = torch.where((order < have[:, None]) & (kept < T), kept, -1).int()
    if own:
        from bit_w4a4_quantized_amd import binding
        s["cache"] = binding.PagedCache(s["k"], s["v"], s["k_scales"], s["v_scales"])
        s["batch"] = binding.PagedBatch(s["table"], s["starts"], s["context"])
    return s


# ------------------------------------------------------------------ one pass
def _turned(x, w, cos, sin, pairs):
    """One of queries or keys [tokens, heads, dim] in fp32; cos, sin [tokens, 1, pairs]."""
    v = x.float()
    if w is not None:
        v = v * (1.0 / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)) * w
    P = cos.shape[-1]
    turned, rest = v[..., : 2 * P], v[..., 2 * P:]
    if pairs == "adjacent":
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = turned[..., :P], turned[..., P:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, rest), -1)


def _places(s, c, slot):
    """Page and offset of cache slots [tokens] or [sequences, n] of the sequences of each row."""
    of = s["of"] if slot.dim() == 1 else torch.arange(slot.shape[0], device=slot.device)[:, None]
    return s["table"][of, slot // c["page"]].long(), slot % c["page"]


def _plain_append(s, c):
    angle = s["positions"].double()[:, _axis_of(s)] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q, k, v = s["new"]
    at = _places(s, c, s["context"][s["of"]].long() + s["at"])
    k, v = _turned(k, s["kw"], cos, sin, c["pairs"]), v.float()
    if c["cache"] in QMAX:
        k, s["k_scales"][at] = _quantized(k, c["cache"])
        v, s["v_scales"][at] = _quantized(v, c["cache"])
    if c["cache"] == "e4m3":        # bytes: indexed writes of the type itself are missing
        s["k"].view(torch.uint8)[at], s["v"].view(torch.uint8)[at] = k.view(torch.uint8), v.view(torch.uint8)
    else:
        s["k"][at], s["v"][at] = k.to(s["k"].dtype), v.to(s["v"].dtype)
    return _turned(q, s["qw"], cos, sin, c["pairs"]).to(q.dtype)


def _axis_of(s):
    n = torch.tensor(s["axes"], device="cuda")
    return torch.repeat_interleave(torch.arange(len(s["axes"]), device="cuda"), n, output_size=sum(s["axes"]))


def _gathered(pages, scales, table):
    """The sequences' cached values [sequences, slots, heads, dim] in fp32."""
    if scales is None:
        return pages[table].flatten(1, 2).float()
    raw = pages.view(torch.uint8)[table].view(pages.dtype)
    return (raw.float() * scales[table][..., None]).flatten(1, 2)


def _plain_attention(s, c):
    B, T, H, G, D, N = c["sequences"], c["tokens"], c["heads"], c["kv_heads"], c["dim"], s["n"]
    table = s["table"].long().clamp_min(0)
    k, v = _gathered(s["k"], s["k_scales"], table), _gathered(s["v"], s["v_scales"], table)
    L = k.shape[1]
    rows = (s["starts"][:-1, None] + torch.arange(T, device="cuda")).clamp_max(N - 1)      # [B, T], padded
    q = s["q"][rows].float().view(B, T, G, H // G, D).transpose(1, 2).reshape(B, G, T * (H // G), D)
    z = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * (1.0 / math.sqrt(D))
    j = torch.arange(L, device="cuda") - s["context"][:, None]                             # [B, L]: drafted token
    i = torch.arange(T, device="cuda")[:, None]
    if s["tree"] is None:
        seen = j[:, None] <= i
    else:
        seen = s["tree"][rows].gather(2, j.clamp(0, s["tree"].shape[1] - 1).long()[:, None].expand(B, T, L))
        seen = (j < 0)[:, None] | (seen & (j < s["starts"].diff()[:, None])[:, None])
    z = z.view(B, G, T, H // G, L).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp_min(-1e38)
    z = z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, G, T * (H // G), L), v.transpose(1, 2).contiguous()).view(B, G, T, H // G, D)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 2, 1, 3, 4).reshape(B, T, H, D)[s["of"], s["at"]].to(s["q"].dtype)


def _plain_keep(s, c):
    path = s["path"].long()
    order = torch.arange(path.shape[1], device="cuda").expand_as(path)
    there = s["context"][:, None].long()
    # a path's end copies its first token onto itself
    src = _places(s, c, there + torch.where(path < 0, path[:, :1], path))
    dst = _places(s, c, there + torch.where(path < 0, path[:, :1], order))
    for t in (s["k"], s["v"], s["k_scales"], s["v_scales"]):
        if t is not None:
            b = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
            b[dst] = b[src]


def _state(s, c):
    """The cache as it is left: 8-bit integers as the values they stand for (the type of the step's tokens)."""
    out = {"k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    for name in ("k", "v"):
        x = s[name]
        out[name] = (x.float() * s[name + "_scales"][..., None]).to(DTYPES[c["dtype"]]) if c["cache"] == "int8" else x
    return out


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "attention":
            return _plain_attention(s, c)
        if c["op"] == "append":
            return {"q": _plain_append(s, c), **_state(s, c)}
        _plain_keep(s, c)
        return _state(s, c)
    from bit_w4a4_quantized_amd import binding
    if c["op"] == "attention":
        return binding.svdq_tree_attention(s["cache"], s["batch"], s["q"], tree=s["tree"])
    if c["op"] == "append":
        q, k, v = s["new"]
        q = binding.svdq_rope_append(s["cache"], s["batch"], q, k, v, s["positions"], s["inv_freq"], s["axes"],
                                     pairs=c["pairs"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS)
        return {"q": q, **_state(s, c)}
    binding.svdq_cache_keep(s["cache"], s["batch"], s["path"])
    return _state(s, c)


# ------------------------------------------------------------------ what a pass cannot do without
def _mean(most, low, ragged):
    return (most + low) / 2 if ragged else most


def work(case):
    c = case
    B, T, H, G, D, b = c["sequences"], c["tokens"], c["heads"], c["kv_heads"], c["dim"], SIZE[c["cache"]]
    row = G * (D * b + (4 if b == 1 else 0))                # keys, or values, of one token in the cache
    tokens = B * _mean(T, max(1, T // 2), c["ragged"])
    past = _mean(c["context"], c["context"] // 2, c["ragged"])
    if c["op"] == "append":
        axes = c["axes"].count(",") + 1
        return {"bytes": tokens * (2 * (2 * H + 2 * G) * D + 2 * row + 4 * axes),
                "flops": tokens * ((7 if c["norm"] else 3) * (H + G) + 2 * G) * D}
    if c["op"] == "keep":
        moved = max(1.0, c["path"] - 1.0) if B == 1 else B * max(0.5, (c["path"] - 1) / 2)
        return {"bytes": moved * 4 * row, "flops": 0}
    seen = past + (tokens / B + 1) / 2
    return {"bytes": B * (past + tokens / B) * 2 * row + 4 * tokens * H * D, "flops": 4 * tokens * H * D * seen}


# ------------------------------------------------------------------ the definitions in 64 bits
def _wide(pages, scales, ids):
    """fp64 values of the pages with these numbers, one behind the other."""
    x = torch.stack([pages[i].float() for i in ids]).double()
    if scales is not None:
        x = x * torch.stack([scales[i] for i in ids]).double()[..., None]
    return x.reshape(-1, *x.shape[2:])


def exact(case, seed):
    s, c = prepare(case, seed), case
    d = lambda t: t.to(torch.float64)  # noqa: E731
    starts, context, table, page = s["starts"].tolist(), s["context"].tolist(), s["table"].tolist(), c["page"]
    G, D = c["kv_heads"], c["dim"]
    if c["op"] == "attention":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        for b in range(c["sequences"]):
            n = starts[b + 1] - starts[b]
            used = table[b][: -(-(context[b] + n) // page)]
            k = _wide(s["k"], s["k_scales"], used)[: context[b] + n]
            v = _wide(s["v"], s["v_scales"], used)[: context[b] + n]
            see = torch.ones(n, context[b] + n, dtype=torch.bool, device="cuda")
            see[:, context[b]:] = torch.ones(n, n, device="cuda").tril() > 0 if s["tree"] is None else \
                s["tree"][starts[b]:starts[b + 1], :n]
            for h in range(c["heads"]):
                g = h // (c["heads"] // G)
                z = torch.mm(d(s["q"][starts[b]:starts[b + 1], h]), k[:, g].T) / math.sqrt(D)
                out[starts[b]:starts[b + 1], h] = torch.softmax(torch.where(see, z, -math.inf), -1) @ v[:, g]
        return out
    out = {"k_scales": None, "v_scales": None}
    if c["op"] == "keep":
        for name in ("k", "v", "k_scales", "v_scales"):
            if s[name] is None:
                continue
            x = s[name].float() if name in ("k", "v") and c["cache"] in QMAX else s[name]
            x, old = d(x), d(x)
            for b, path in enumerate(s["path"].tolist()):
                for i, j in enumerate(path):
                    if j >= 0:
                        at, to = context[b] + j, context[b] + i
                        x[table[b][to // page], to % page] = old[table[b][at // page], at % page]
            out[name] = x
        if c["cache"] == "int8":
            for name in ("k", "v"):
                out[name] = out[name] * out[name + "_scales"][..., None]
        return out
    # append: each pair as a complex number, multiplied by exp(i angle)
    at = sum(([i] * n for i, n in enumerate(s["axes"])), [])
    angle = d(s["positions"])[:, at] * d(s["inv_freq"])
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    P = angle.shape[-1]
    low = slice(0, 2 * P, 2) if c["pairs"] == "adjacent" else slice(0, P)
    high = slice(1, 2 * P, 2) if c["pairs"] == "adjacent" else slice(P, 2 * P)
    new = [d(t) for t in s["new"]]
    for i, w in enumerate((s["qw"], s["kw"])):
        x = new[i] if w is None else new[i] / (new[i].pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * d(w)
        y = x.clone()
        z = torch.complex(x[..., low].contiguous(), x[..., high].contiguous()) * turn
        y[..., low], y[..., high] = z.real, z.imag
        new[i] = y
    out["q"] = new[0]
    places = [(b, i) for b in range(c["sequences"]) for i in range(starts[b + 1] - starts[b])]
    pages = torch.tensor([table[b][(context[b] + i) // page] for b, i in places], device="cuda")
    rest = torch.tensor([(context[b] + i) % page for b, i in places], device="cuda")
    for name, x in (("k", new[1]), ("v", new[2])):
        old = d(s[name].float() if c["cache"] in QMAX else s[name])
        if c["cache"] in QMAX:
            top = x.abs().max(-1).values.clamp_min(TINY)
            scales = d(s[name + "_scales"])
            if c["cache"] == "int8":
                x = torch.round(x * 127.0 / top[..., None]) * (top / 127.0)[..., None]
                old = old * scales[..., None]
            else:
                x = x / top[..., None] * 448.0
            scales[pages, rest] = top / QMAX[c["cache"]]
            out[name + "_scales"] = scales
        old[pages, rest] = x
        out[name] = old
    return out
