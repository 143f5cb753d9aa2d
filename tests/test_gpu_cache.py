"""The operators around a paged cache against plain 64-bit implementations: svdq_rope_append,
svdq_tree_attention, svdq_cache_keep.

Tolerances are derived as in test_gpu_block.py: U is half a step of a 16-bit type relative to the value,
EPS32 the fp32 rounding unit."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_w4a4_quantized_amd import binding  # noqa: E402
from test_gpu_block import BF16, E4M3, EPS32, F16, F64, SMALL, TINY, U, check, gen, randn, rope64  # noqa: E402

I8 = torch.int8
QMAX = {I8: 127.0, E4M3: 448.0}
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.lib()
    yield
    torch.cuda.synchronize()


def quantized(v, dtype):
    a = v.abs().amax(-1).clamp_min(TINY)
    c = v * (QMAX[dtype] / a)[..., None]
    return (c.round().to(I8) if dtype is I8 else c.to(E4M3)), a / QMAX[dtype]


def raw(t):
    """Bytes of a tensor whose type lacks what a test needs of it."""
    return t.view(torch.uint8) if t.dtype is E4M3 else t


class Pages:
    """A cache on the host and its copy on the device, in pages handed out in a mixed order."""

    def __init__(self, g, counts, contexts, heads, dim, cache, page, spare=2, heads_first=False, pad=0, width=None):
        B = len(counts)
        need = [-(-(c + n) // page) for c, n in zip(contexts, counts)]
        self.width = max(need + [1]) if width is None else width
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        self.table = torch.full((B, self.width), -1, dtype=torch.int32)
        for b in range(B):
            for i in range(min(need[b], self.width)):
                self.table[b, i] = order.pop()
        self.page, self.heads, self.dim, self.type, self.contexts, self.counts = page, heads, dim, cache, contexts, counts
        starts = [0]
        for n in counts:
            starts.append(starts[-1] + n)
        self.starts, self.tokens = starts, starts[-1]
        self.host, self.dev = {}, {}
        for name in ("k", "v"):
            x = randn(g, self.pages, page, heads, dim)
            x[..., 0] *= 5
            if cache in QMAX:
                self.host[name], self.host[name + "_scales"] = quantized(x, cache)
            else:
                self.host[name], self.host[name + "_scales"] = x.to(cache), None
        # heads_first: pages keep a head's tokens together; pad: unused bytes behind a token's heads
        for name, t in self.host.items():
            if t is None:
                self.dev[name] = None
            elif name.endswith("scales"):
                self.dev[name] = t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if heads_first else t.cuda()
            else:
                b = raw(t)
                if heads_first:
                    d = b.transpose(1, 2).contiguous().cuda().transpose(1, 2)
                else:
                    d = torch.zeros(self.pages, page, heads, dim + pad, dtype=b.dtype, device="cuda")[..., :dim]
                    d.copy_(b)
                self.dev[name] = d.view(t.dtype)
        self.upload()

    def upload(self):
        self.cache = binding.PagedCache(self.dev["k"], self.dev["v"], self.dev["k_scales"], self.dev["v_scales"])
        self.batch = binding.PagedBatch(self.table.cuda(), torch.tensor(self.starts, dtype=torch.int32).cuda(),
                                        torch.tensor(self.contexts, dtype=torch.int32).cuda())

    def values(self, name, b, n):
        """fp64 [n, heads, dim] of sequence b's slots and which of them exist."""
        slot = torch.arange(n)
        col = slot // self.page
        id_ = torch.where(col < self.width, self.table[b][col.clamp_max(self.width - 1)].long(), -1)
        there = (id_ >= 0) & (id_ < self.pages)
        at = id_.clamp(0, self.pages - 1)
        x = raw(self.host[name])[at, slot % self.page].view(self.host[name].dtype).to(F64)
        if self.host[name + "_scales"] is not None:
            x = x * self.host[name + "_scales"][at, slot % self.page].to(F64)[..., None]
        return x, there


def attention64(p, q, tree, scale, up):
    """Outputs and their tolerances, fp64; rows of no sequence: zeros."""
    H, D = q.shape[1], q.shape[2]
    group = H // p.heads
    out, tol = torch.zeros(q.shape, dtype=F64), torch.zeros(q.shape, dtype=F64)
    for b, (n, ctx) in enumerate(zip(p.counts, p.contexts)):
        if n == 0:
            continue
        s0 = p.starts[b]
        k, there = p.values("k", b, ctx + n)
        v, _ = p.values("v", b, ctx + n)
        see = torch.ones(n, ctx + n, dtype=torch.bool)
        if tree is None:
            see[:, ctx:] = torch.ones(n, n).tril().bool()
        else:
            w = min(n, tree.shape[1])
            see[:, ctx:] = False
            see[:, ctx:ctx + w] = tree[s0:s0 + n, :w].bool()
        see &= there
        for h in range(H):
            qq = q[s0:s0 + n, h].to(F64)
            kk, vv = k[:, h // group].clone(), v[:, h // group].clone()
            seen_any = see.any(0)
            kk[~seen_any], vv[~seen_any] = 0, 0
            z = (qq @ kk.T) * scale
            size = (qq.abs() @ kk.abs().T) * scale                 # of the products a logit sums
            z = torch.where(see, z, torch.tensor(-INF, dtype=F64))
            top = z.amax(-1, keepdim=True)
            e = torch.where(see, torch.exp(z - torch.where(top == -INF, 0, top)), 0)
            l = e.sum(-1, keepdim=True)
            pr = torch.where(l > 0, e / l, 0)
            # rows of V that a row does not see keep out, whatever they hold
            o, a = torch.zeros(n, D, dtype=F64), torch.zeros(n, D, dtype=F64)
            for i in range(n):
                o[i] = pr[i, see[i]] @ vv[see[i]]
                a[i] = pr[i, see[i]] @ vv[see[i]].abs()
            out[s0:s0 + n, h] = o
            # a logit's sum, its products with scales, the power's argument (twice: the maximum's too)
            zs = torch.where(see, size, 0).amax(-1, keepdim=True)
            dz = 2 * (2 * D + 8) * EPS32 * zs
            rel = up + 2 * dz + (ctx + n + 16) * 2 * EPS32
            tol[s0:s0 + n, h] = a * rel * 1.01 + U[q.dtype] * 1.001 * o.abs() + SMALL[q.dtype]
            if p.type in QMAX:          # fp16 products of probability and scale below its range: 2^-25 of the largest
                tol[s0:s0 + n, h] += (ctx + n) * 2.0 ** -25 * torch.nan_to_num(vv.abs(), 0, 0, 0).amax()
    return out, tol


def random_tree(g, counts, width=None):
    """Rows of packed tokens: each token hangs from any before it, and sees itself and its ancestors."""
    W = max(counts + [1]) if width is None else width
    rows = []
    for n in counts:
        sees = torch.zeros(n, max(n, W), dtype=torch.bool)
        for i in range(n):
            if i:
                sees[i] = sees[int(torch.randint(0, i, (1,), generator=g))]
            sees[i, i] = True
        rows.append(sees[:, :W])
    return torch.cat(rows) if rows else torch.zeros(0, W, dtype=torch.bool)


def attend(p, q, tree, scale=None, workspace=None, behind=0, q_pad=0, own_out=True):
    """The operator's result on strided queries, into a guarded buffer with rows of no sequence behind."""
    N, H, D = q.shape
    buf = torch.full((N + behind, H * D + q_pad), 3.0, dtype=q.dtype)
    buf[:N, :H * D] = q.reshape(N, H * D)
    qd = buf.cuda()[:, :H * D].unflatten(-1, (H, D))
    if tree is not None:
        tree = torch.cat([tree, torch.ones(behind, tree.shape[1], dtype=tree.dtype)]).cuda()
    if not own_out:
        return binding.svdq_tree_attention(p.cache, p.batch, qd, tree, scale, workspace=workspace)[:N].cpu()
    ob = torch.full((N + behind + 2, H, D + 8), 72.0, dtype=q.dtype, device="cuda")
    out = ob[1:1 + N + behind, :, :D]
    got = binding.svdq_tree_attention(p.cache, p.batch, qd, tree, scale, out=out, workspace=workspace)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr()
    o = ob.float().cpu()
    assert (o[0] == 72).all() and (o[1 + N:] == 72).all() and (o[..., D:] == 72).all()
    return out[:N].cpu()


def attention_case(counts, contexts, heads, kv, dim, dtype, cache, page, tree, seed=0, scale=None, **kw):
    g = gen(seed + dim + page + sum(counts))
    more = {n: kw.pop(n) for n in ("heads_first", "pad", "width") if n in kw}
    p = Pages(g, counts, contexts, kv, dim, cache, page, **more)
    q = (2 * randn(g, p.tokens, heads, dim)).to(dtype)
    t = random_tree(g, counts) if tree else None
    got = attend(p, q, t, scale, **kw)
    up = U[F16] if cache in QMAX else U[dtype]
    want, tol = attention64(p, q, t, dim ** -0.5 if scale is None else scale, up)
    check(got, want, tol, f"attention {counts} over {contexts} {heads}/{kv}x{dim} {dtype} {cache} page {page}")


KINDS = [(F16, F16), (BF16, BF16), (F16, I8), (BF16, I8), (F16, E4M3), (BF16, E4M3)]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
def test_attention_types(dtype, cache, dim):
    attention_case([1, 5, 1], [40, 7, 130], 4, 2, dim, dtype, cache, 16, True, behind=2, q_pad=8)
    attention_case([3, 1], [0, 65], 2, 2, dim, dtype, cache, 32, False, seed=1)


@pytest.mark.parametrize("dim", [8, 24, 72, 104, 136, 200])
def test_attention_odd_dims(dim):
    attention_case([2, 4], [33, 1], 6, 2, dim, F16, F16, 8, True, q_pad=3)
    attention_case([2, 4], [33, 1], 6, 2, dim, BF16, BF16, 64, False, pad=8)


@pytest.mark.parametrize("page", [1, 2, 8, 64, 256, 4096])
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 1), (24, 8), (17, 1), (40, 2)])
def test_attention_pages_and_groups(page, heads, kv):
    attention_case([4, 1, 9], [31, 33, 0], heads, kv, 64, F16, F16, page, True, heads_first=page % 16 == 0)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 61, 64, 65, 100, 130, 200])
def test_attention_token_counts(n):
    attention_case([n, 1, n // 2 + 1], [70, 3, 129], 4, 4, 64, BF16, BF16, 16, True)
    attention_case([n], [65], 8, 2, 128, F16, I8, 64, False, seed=2)


@pytest.mark.parametrize("keys", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1023, 1025])
def test_attention_lengths(keys):
    attention_case([1], [keys - 1], 4, 2, 64, F16, F16, 32, False)
    attention_case([1, 2], [keys - 1, keys // 2], 4, 1, 128, BF16, E4M3, 8, True)


def test_attention_long():
    """Split over the length, joined; with less room than asked for, and with none."""
    g = gen(3)
    p = Pages(g, [1, 3], [20011, 4000], 2, 64, F16, 64)
    q = (2 * randn(g, 4, 4, 64)).to(F16)
    need = binding.tree_attention_workspace_bytes(2, 4, 4, 2, 64, p.width, 64)
    assert need > 0
    want, tol = attention64(p, q, None, 0.125, U[F16])
    results = []
    for room in (need, need // 3, 16):
        ws = torch.full((room + 64,), 123, dtype=torch.uint8, device="cuda")
        results.append(attend(p, q, None, workspace=ws[:room]))
        assert bool((ws[room:] == 123).all())
        check(results[-1], want, tol, f"long, room {room}")
    assert torch.equal(results[0], attend(p, q, None, own_out=False))


def test_attention_many_sequences():
    """More than the 64 sequences that one look takes in, and more than 64 looks' worth; some without tokens."""
    for B in (65, 200, 4200):
        counts = [0 if b % 7 == 3 else 1 + b % 2 for b in range(B)]
        attention_case(counts, [b % 9 for b in range(B)], 2, 1, 64, F16, F16, 8, False, seed=B)


def test_attention_empty_rows():
    """Rows that see nothing are zeros: no context and an empty row of the tree, a column past the width, absent pages."""
    g = gen(8)
    p = Pages(g, [3, 2, 4, 1], [0, 5, 0, 0], 2, 64, F16, 8)
    q = randn(g, 10, 4, 64).to(F16)
    tree = torch.zeros(10, 2, dtype=torch.uint8)
    tree[1, 0] = tree[4, 1] = 255
    tree[6] = 1
    p.table[3] = -1
    p.upload()
    got = attend(p, q, tree)
    want, tol = attention64(p, q, tree, 0.125, U[F16])
    check(got, want, tol, "empty rows")
    for row in (0, 2, 5, 7, 8, 9):
        assert bool((got[row] == 0).all())
    assert bool((attend(p, q, tree[:, :0]) == 0)[[0, 1, 2, 5, 6, 7, 8, 9]].all())


@pytest.mark.parametrize("rows", [1, 40, 150])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_attention_hidden_values(dtype, cache, rows):
    """Infinities and NaN where no row looks, or some rows do not: unwritten slots, absent pages, siblings in the tree.
    Rows that do see one get infinities and NaN."""
    g = gen(11)
    n = max(rows, 3)
    p = Pages(g, [n, 2], [45, 3], 2, 64, cache, 16, spare=3)
    q = randn(g, n + 2, 2, 64).to(dtype)
    tree = random_tree(g, [n, 2])
    tree[:, 2] = False
    tree[2, 2] = True                        # token 2 of the first sequence is seen by itself alone
    used = torch.zeros(p.pages, 16, dtype=torch.bool)
    for b, m in enumerate((45 + n, 5)):
        for s in range(m):
            used[int(p.table[b, s // 16]), s % 16] = True
    sick = used.logical_not()
    sick[int(p.table[0, 47 // 16]), 47 % 16] = True
    want, tol = attention64(p, q, tree, 0.125, U[F16] if cache in QMAX else U[dtype])
    for name in ("k", "v"):
        if cache in QMAX:
            p.dev[name + "_scales"][sick.cuda()] = NAN if name == "k" else INF
        if cache is E4M3:
            raw(p.dev[name])[sick.cuda()] = 0x7F
        elif cache is not I8:
            p.dev[name][sick.cuda()] = torch.tensor([INF, NAN, -INF, 1.0] * 16).to(cache).cuda()
    got = attend(p, q, tree)
    check(torch.cat([got[:2], got[3:]]), torch.cat([want[:2], want[3:]]), torch.cat([tol[:2], tol[3:]]), "hidden values")
    assert not bool(torch.isfinite(got[2]).all())


def test_attention_bad_pages():
    """Entries that are no pages, and a table shorter than the context, hide their slots."""
    g = gen(12)
    p = Pages(g, [2, 3], [60, 50], 2, 64, F16, 8)
    p.table[0, 2], p.table[0, 5], p.table[1, 0], p.table[1, 3] = p.pages, -7, 2 ** 31 - 1, -2 ** 31
    p.upload()
    q = randn(g, 5, 4, 64).to(F16)
    want, tol = attention64(p, q, None, 0.125, U[F16])
    check(attend(p, q, None), want, tol, "bad pages")
    p.table, p.width = p.table[:, :4].contiguous(), 4
    p.upload()
    want, tol = attention64(p, q, None, 0.125, U[F16])
    check(attend(p, q, None), want, tol, "short table")


@pytest.mark.parametrize("cache", [F16, BF16, I8, E4M3])
def test_attention_large_logits(cache):
    """Logits far apart and a rising maximum: probabilities of 0 and 1, the reference moves many times."""
    g = gen(13)
    dtype = BF16 if cache is BF16 else F16
    p = Pages(g, [2], [700], 1, 64, cache, 32)
    q = torch.zeros(2, 1, 64, dtype=dtype)
    q[..., 0] = 40.0
    got = attend(p, q, None)
    want, tol = attention64(p, q, None, 0.125, U[F16] if cache in QMAX else U[dtype])
    check(got, want, tol, "large logits")


def test_attention_bf16_queries_of_any_size():
    """bf16 queries past fp16's range, and far below it, over a cache of codes."""
    g = gen(14)
    p = Pages(g, [4], [50], 1, 64, I8, 16)
    q = randn(g, 4, 2, 64)
    q = (q * torch.tensor([2.0 ** 100, 2.0 ** -100, 2.0 ** 20, 0.0])[:, None, None]).to(BF16)
    for row, scale in ((0, 2.0 ** -103), (1, 2.0 ** 97), (2, 2.0 ** -23), (3, 1.0)):
        got = attend(p, q, None, scale=scale)
        want, tol = attention64(p, q, None, scale, U[F16])
        check(got[row], want[row], tol[row], f"row {row}")


def test_attention_scales_far_apart():
    """V's scales over many orders within a sequence: the reference they are taken relative to moves."""
    g = gen(15)
    for cache in (I8, E4M3):
        p = Pages(g, [1], [400], 1, 64, cache, 16)
        s = 10.0 ** (torch.rand(p.pages, 16, 1, generator=g) * 12 - 6)
        p.host["v_scales"] = (p.host["v_scales"] * s).float()
        p.dev["v_scales"].copy_(p.host["v_scales"])
        q = randn(g, 1, 2, 64).to(F16)
        want, tol = attention64(p, q, None, 1.0, U[F16])
        got = attend(p, q.to(BF16), None, scale=1.0)      # fp16 outputs could overflow
        want, tol = attention64(p, q.to(BF16), None, 1.0, U[F16])
        check(got, want, tol, "scales")
        p.dev["v_scales"].zero_()
        assert bool((attend(p, q, None) == 0).all())


def test_attention_same_bits():
    g = gen(16)
    for cache, n in ((F16, 1), (I8, 1), (BF16, 70), (E4M3, 200)):
        p = Pages(g, [n, n], [900, 300], 2, 128, cache, 16)
        q = randn(g, 2 * n, 4, 128).to(BF16 if cache is BF16 else F16)
        r = [attend(p, q, None) for _ in range(3)]
        assert torch.equal(r[0], r[1]) and torch.equal(r[0], r[2])


def test_attention_in_place_and_empty():
    g = gen(17)
    p = Pages(g, [2, 5], [40, 9], 2, 128, F16, 16)
    q = randn(g, 7, 4, 128).to(F16).cuda()
    want = binding.svdq_tree_attention(p.cache, p.batch, q)
    x = q.clone()
    assert binding.svdq_tree_attention(p.cache, p.batch, x, out=x).data_ptr() == x.data_ptr()
    assert torch.equal(x, want)
    none = binding.PagedBatch(p.batch.page_table[:0], p.batch.starts[:1], p.batch.context[:0])
    out = torch.full_like(q, 5.0)
    binding.svdq_tree_attention(p.cache, none, q, out=out)
    assert bool((out == 5).all())
    assert binding.svdq_tree_attention(p.cache, p.batch, q[:0]).shape == (0, 4, 128)


def test_attention_far_offsets():
    """Elements past 2^32 bytes from the first page's start."""
    pages = (1 << 32) // (2 * 64 * 64 * 2) + 70
    g = gen(18)
    p = Pages(g, [2], [200], 2, 64, F16, 64)
    k = torch.zeros(pages, 64, 2 * 64, dtype=F16, device="cuda").view(pages, 64, 2, 64)
    v = torch.zeros_like(k)
    ids = [pages - 1 - 3 * i for i in range(p.width)]
    for i, id_ in enumerate(ids):
        k[id_], v[id_] = p.dev["k"][int(p.table[0, i])], p.dev["v"][int(p.table[0, i])]
    q = randn(g, 2, 4, 64).to(F16)
    want, tol = attention64(p, q, None, 0.125, U[F16])
    p.table = torch.tensor([ids], dtype=torch.int32)
    p.dev["k"], p.dev["v"] = k, v
    p.upload()
    check(attend(p, q, None), want, tol, "far offsets")


# ------------------------------------------------------------------ appending
def append_case(counts, contexts, heads, kv, dim, dtype, cache, page, axis_pairs, pairs, norm, seed=0, pad=0, odd=0,
                queries=True, behind=1, far=1, heads_first=False):
    g = gen(seed + dim + sum(counts))
    p = Pages(g, counts, contexts, kv, dim, cache, page, heads_first=heads_first)
    N = p.tokens + behind
    rows = randn(g, N, (heads + 2 * kv) * dim + pad + odd).to(dtype)
    x = rows[:, odd:odd + (heads + 2 * kv) * dim]
    split = lambda t: [u.unflatten(-1, (-1, dim)) for u in t[:, odd:odd + (heads + 2 * kv) * dim].split(  # noqa: E731
        [heads * dim, kv * dim, kv * dim], -1)]
    q, k, v = split(rows)
    pos = torch.randint(0, 300 * far, (N, len(axis_pairs)), generator=g, dtype=torch.int32)
    freq = torch.cat([10000.0 ** (-torch.arange(n, dtype=F64) / max(n, 1)) for n in axis_pairs]).float()
    qw, kw = (1 + 0.2 * randn(g, dim), 1 + 0.2 * randn(g, dim)) if norm else (None, None)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    dev = rows.cuda()
    qd, kd, vd = split(dev)
    got = binding.svdq_rope_append(p.cache, p.batch, qd if queries else None, kd, vd, pos.cuda(), freq.cuda(), axis_pairs,
                                   pairs, cu(qw) if queries else None, cu(kw))
    torch.cuda.synchronize()
    assert torch.equal(dev.cpu(), rows)      # the packed projection is only read
    turned = {}
    for name, t, w in (("q", q, qw), ("k", k, kw)):
        want, size = rope64(t, w, pos, freq, axis_pairs, pairs, 1e-6, False)
        turned[name] = want, (2.0 ** -20 + (dim / 8 + 8) * EPS32) * size
    if queries:
        want, err = turned["q"]
        check(got, want, U[dtype] * 1.001 * want.abs() + err + SMALL[dtype], "queries")
    turned["v"] = v.to(F64), torch.zeros(v.shape, dtype=F64)
    for name in ("k", "v"):
        new, err = turned[name]
        after = p.dev[name].cpu()
        scales = None if cache not in QMAX else p.dev[name + "_scales"].cpu()
        touched = torch.zeros(p.pages, page, dtype=torch.bool)
        for b, (n, ctx) in enumerate(zip(counts, contexts)):
            for i in range(n):
                slot = ctx + i
                id_ = int(p.table[b, slot // page]) if slot // page < p.width else -1
                if not 0 <= id_ < p.pages:
                    continue
                touched[id_, slot % page] = True
                t = p.starts[b] + i
                u, e = new[t], err[t]
                at = (id_, slot % page)
                if cache not in QMAX:
                    check(raw(after)[at], u, U[cache] * 1.001 * u.abs() + e + (SMALL[cache] if name == "k" else 0), name)
                    continue
                a = u.abs().amax(-1).clamp_min(TINY)
                ea = e.amax(-1)
                s = scales[at].to(F64)
                check(s, a / QMAX[cache], (ea + 4 * EPS32 * a) / QMAX[cache], name + " scales")
                c = raw(after)[at].view(cache).to(F64)
                exact = u / a[:, None] * QMAX[cache]
                off = (e / a[:, None] + (ea / a)[:, None] + 4 * EPS32) * QMAX[cache]
                half = 0.5 if cache is I8 else torch.maximum(exact.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=F64))
                check(c, exact, half + off * 1.1, name + " codes")
        for t, old in ((raw(after), raw(p.host[name])), (scales, p.host[name + "_scales"])):
            if t is not None:
                assert torch.equal(t[~touched], old[~touched]), "a slot of no token was written"
    return p


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("dim,axis_pairs", [(64, (32,)), (80, (10, 14, 16)), (128, (8, 28, 28)), (128, (16, 16)), (256, (128,)),
                                            (96, (0, 24)), (16, (3,)), (208, (100, 4))])
def test_append(dim, axis_pairs, pairs, dtype, cache):
    append_case([1, 5, 0, 3], [40, 7, 9, 0], 3, 2, dim, dtype, cache, 8, axis_pairs, pairs, dim != 64)
    append_case([4], [0], 4, 1, dim, dtype, cache, 64, axis_pairs, pairs, False, pad=8, heads_first=True, queries=dim != 80)


@pytest.mark.parametrize("dim", [8, 24, 72, 104])
def test_append_odd_dims_and_rows(dim):
    for pairs in ("adjacent", "halves"):
        append_case([2, 7], [5, 1], 2, 1, dim, F16, F16, 16, (dim // 4, dim // 4), pairs, True, odd=1)
        append_case([2, 7], [5, 1], 2, 1, dim, BF16, BF16, 16, (dim // 4,), pairs, True, pad=3)


@pytest.mark.parametrize("heads,kv", [(1, 1), (2, 1), (32, 8), (5, 5), (40, 1), (3, 70)])
def test_append_head_counts(heads, kv):
    append_case([1], [33], heads, kv, 64, F16, E4M3, 16, (32,), "halves", False)
    append_case([6, 1], [0, 90], heads, kv, 32, BF16, I8, 16, (16,), "adjacent", True)


@pytest.mark.parametrize("heads,kv,dim", [(1, 1, 64), (2, 1, 32), (4, 2, 80)])
def test_append_several_tokens_a_wave(heads, kv, dim):
    """Thousands of tokens of few heads: a wave has several, of several sequences."""
    counts = [1 + (b * 7) % 5 for b in range(1500)]
    append_case(counts, [b % 3 for b in range(1500)], heads, kv, dim, F16, F16, 4, (dim // 2,), "halves", True, behind=5)


def test_append_values_of_zero_and_far_positions():
    p = append_case([3], [2], 2, 2, 64, F16, I8, 8, (32,), "halves", False, far=10 ** 6)
    zero = torch.zeros(3, 2, 64, dtype=F16, device="cuda")
    pos, freq = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda")
    binding.svdq_rope_append(p.cache, p.batch, None, zero, zero, pos, freq, (32,))
    at = [(int(p.table[0, s // 8]), s % 8) for s in (2, 3, 4)]
    for name in ("k", "v"):
        for i in at:
            assert bool((p.dev[name][i] == 0).all()) and bool((p.dev[name + "_scales"][i] == TINY / 127).all())


def test_append_in_place_and_bad_pages():
    """Queries turned in place; tokens whose slot has no page are turned and go nowhere."""
    g = gen(21)
    p = Pages(g, [3, 2], [6, 30], 2, 64, BF16, 8)
    p.table[0, 1], p.table[1, 3] = -1, p.pages
    p.upload()
    q, k, v = (randn(g, 5, n, 64).to(BF16).cuda() for n in (4, 2, 2))
    pos = torch.arange(5, dtype=torch.int32, device="cuda")[:, None].contiguous()
    freq = torch.ones(32, device="cuda") * 0.1
    want, kept = binding.svdq_rope_axes(q, k, pos, freq, (32,), pairs="halves")
    got = binding.svdq_rope_append(p.cache, p.batch, q, k, v, pos, freq, (32,), pairs="halves", q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)
    after = p.dev["k"].cpu()
    for t, (b, s) in enumerate([(0, 6), (0, 7), (0, 8), (1, 30), (1, 31)]):
        id_ = int(p.table[b, s // 8])
        if 0 <= id_ < p.pages:
            assert torch.equal(after[id_, s % 8], kept[t].cpu())
            after[id_, s % 8] = p.host["k"][id_, s % 8]
    assert torch.equal(after, p.host["k"])
    short = binding.PagedBatch(p.batch.page_table[:, :0], p.batch.starts, p.batch.context)
    binding.svdq_rope_append(p.cache, short, q, k, v, pos, freq, (32,))
    none = binding.PagedBatch(p.batch.page_table[:0], p.batch.starts[:1], p.batch.context[:0])
    binding.svdq_rope_append(p.cache, none, q, k, v, pos, freq, (32,))
    assert binding.svdq_rope_append(p.cache, p.batch, q[:0], k[:0], v[:0], pos[:0], freq, (32,)).shape == (0, 4, 64)


# ------------------------------------------------------------------ keeping
@pytest.mark.parametrize("cache", [F16, BF16, I8, E4M3])
@pytest.mark.parametrize("page,heads,dim,heads_first", [(8, 3, 80, False), (64, 1, 128, True), (1, 2, 256, False)])
def test_keep(cache, page, heads, dim, heads_first):
    g = gen(31)
    counts, contexts = [9, 30, 1, 64, 5, 0], [11, 0, 8, 62, 3, 4]
    p = Pages(g, counts, contexts, heads, dim, cache, page, heads_first=heads_first)
    p.table[4, (3 + 3) // page] = -1         # sequence 4's fourth token has no page
    p.upload()
    path = torch.full((6, 20), -1, dtype=torch.int32)
    path[0, :4] = torch.tensor([0, 1, 5, 8])
    path[1, :3] = torch.tensor([2, 3, 29])
    path[2, 0] = 0
    path[3, :20] = torch.arange(20) * 3 + 1
    path[4, :5] = torch.tensor([1, 2, 3, 4, 5])      # one past its tokens: left out
    path[5, :2] = torch.tensor([0, 1])
    want = {n: None if t is None else raw(t).clone() for n, t in p.host.items()}
    for b in range(6):
        old = {n: None if t is None else t.clone() for n, t in want.items()}
        for i, j in enumerate(path[b].tolist()):
            if j < 0 or j >= counts[b] or i >= counts[b]:
                continue
            ids = [int(p.table[b, (contexts[b] + s) // page]) for s in (j, i)]
            if min(ids) < 0:
                continue
            for n, t in want.items():
                if t is not None:
                    t[ids[1], (contexts[b] + i) % page] = old[n][ids[0], (contexts[b] + j) % page]
    wide = torch.full((6, 23), 7, dtype=torch.int32)
    wide[:, :20] = path
    binding.svdq_cache_keep(p.cache, p.batch, wide.cuda()[:, :20])
    for n, t in want.items():
        if t is not None:
            assert torch.equal(raw(p.dev[n]).cpu(), t), n
    binding.svdq_cache_keep(p.cache, p.batch, wide.cuda()[:, :0])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("cache", [F16, I8])
def test_draft_checked_and_kept(cache):
    """A tree of drafted tokens appended, checked and its accepted path kept leaves what decoding the path alone
    leaves: the next token's attention agrees, and the tree's rows agree with a chain over the path."""
    g = gen(41)
    kv, heads, dim, ctx = 2, 4, 64, 37
    parent = [-1, 0, 0, 1, 2, 4, 4, 5]
    path = [0, 2, 4, 5]
    n = len(parent)
    tree = torch.zeros(n, n, dtype=torch.bool)
    depth = [0] * n
    for i, up in enumerate(parent):
        if up >= 0:
            tree[i], depth[i] = tree[up], depth[up] + 1
        tree[i, i] = True
    q, k, v = (randn(g, n + 1, h, dim).to(F16) for h in (heads, kv, kv))
    freq = (100.0 ** (-torch.arange(32) / 32)).cuda()
    runs = []
    for drafted in (True, False):
        p = Pages(gen(5), [n], [ctx], kv, dim, cache, 16)
        rows = list(range(n)) if drafted else path
        pos = torch.tensor([[ctx + depth[i]] for i in rows], dtype=torch.int32).cuda()
        starts = torch.tensor([0, len(rows)], dtype=torch.int32).cuda()
        batch = binding.PagedBatch(p.table.cuda(), starts, torch.tensor([ctx], dtype=torch.int32).cuda())
        turned = binding.svdq_rope_append(p.cache, batch, q[rows].cuda(), k[rows].cuda(), v[rows].cuda(), pos, freq, (32,))
        o = binding.svdq_tree_attention(p.cache, batch, turned, tree=tree.cuda() if drafted else None)
        if drafted:
            o = o[path]
            binding.svdq_cache_keep(p.cache, batch, torch.tensor([path + [-1]], dtype=torch.int32).cuda())
        after = binding.PagedBatch(p.table.cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda(),
                                   torch.tensor([ctx + len(path)], dtype=torch.int32).cuda())
        turned = binding.svdq_rope_append(p.cache, after, q[n:].cuda(), k[n:].cuda(), v[n:].cuda(),
                                          torch.tensor([[ctx + len(path)]], dtype=torch.int32).cuda(), freq, (32,))
        runs.append((o.cpu(), binding.svdq_tree_attention(p.cache, after, turned).cpu()))
    (a, x), (b, y) = runs
    assert torch.equal(x, y)                 # the same cache, the same call
    # the same terms in another order and at other places of a tile: two results within their own errors
    check(a, b.to(F64), 2 * (U[F16] * 2 + 200 * EPS32) * 8 + SMALL[F16], "rows of the tree")


def test_captured_and_replayed():
    """The three operators in one graph, replayed with new contents and other work in between."""
    g = gen(51)
    p = Pages(g, [3, 2], [100, 700], 2, 64, E4M3, 16, spare=4)
    q, k, v = (randn(g, 5, h, 64).to(F16).cuda() for h in (4, 2, 2))
    pos = torch.arange(5, dtype=torch.int32, device="cuda")[:, None].contiguous()
    freq = torch.full((32,), 0.05, device="cuda")
    path = torch.tensor([[1, 2], [0, -1]], dtype=torch.int32).cuda()
    tree = random_tree(g, [3, 2]).cuda()

    def step():
        t = binding.svdq_rope_append(p.cache, p.batch, q, k, v, pos, freq, (32,))
        o = binding.svdq_tree_attention(p.cache, p.batch, t, tree=tree)
        binding.svdq_cache_keep(p.cache, p.batch, path)
        return o

    start = {n: t.clone() for n, t in p.dev.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        for t, h in ((q, 4), (k, 2), (v, 2)):
            t.copy_(randn(g, 5, h, 64).to(F16))
        p.batch.context.copy_(torch.tensor([100 - i, 700 - 50 * i], dtype=torch.int32))
        for n, t in p.dev.items():
            raw(t).copy_(raw(start[n]))
        eager = step().clone()
        state = {n: raw(t).clone() for n, t in p.dev.items()}
        for n, t in p.dev.items():
            raw(t).copy_(raw(start[n]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        for n, t in p.dev.items():
            assert torch.equal(raw(t), state[n])


def test_on_another_stream():
    g = gen(52)
    p = Pages(g, [2, 2], [900, 300], 2, 64, F16, 16)
    q, k, v = (randn(g, 4, h, 64).to(F16).cuda() for h in (4, 2, 2))
    pos = torch.arange(4, dtype=torch.int32, device="cuda")[:, None].contiguous()
    freq = torch.full((32,), 0.05, device="cuda")
    t0 = binding.svdq_rope_append(p.cache, p.batch, q, k, v, pos, freq, (32,))
    o0 = binding.svdq_tree_attention(p.cache, p.batch, t0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        t1 = binding.svdq_rope_append(p.cache, p.batch, q, k, v, pos, freq, (32,), stream=side.cuda_stream)
        o1 = binding.svdq_tree_attention(p.cache, p.batch, t1, stream=side.cuda_stream)
        binding.svdq_cache_keep(p.cache, p.batch, torch.tensor([[0], [0]], dtype=torch.int32).cuda(), stream=side.cuda_stream)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(t0, t1) and torch.equal(o0, o1)
        torch.cuda.synchronize()
