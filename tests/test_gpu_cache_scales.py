"""svdq_tree_attention over 8-bit caches whose scales of V differ by any factor: what a row does not see, or sees with next
to no probability, leaves its other terms alone.

The tolerance is a row's own.  A product of probability and scale is rounded to fp16 relative to the largest that the row
has seen, which lies at 1 or above: half a step (2^-11) of itself, 2^-25 of that largest below fp16's normal range.  Its
code is at most qmax."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from strict import check  # noqa: E402
from test_gpu_cache import (BF16, E4M3, EPS32, F16, F64, I8, QMAX, SMALL, U, Pages, _gpu, attend, gen,  # noqa: E402, F401
                            randn, random_tree)

INF = math.inf


def own64(p, q, see, scale):
    """Of one sequence, each row from the keys that it sees alone: outputs and tolerances."""
    n, H, D = q.shape
    keys = see.shape[1]
    k, v = p.values("k", 0, keys)[0], p.values("v", 0, keys)[0]
    s = p.values_of_scales(keys)
    out, tol = torch.zeros(q.shape, dtype=F64), torch.zeros(q.shape, dtype=F64)
    for h in range(H):
        g = h // (H // p.heads)
        for i in range(n):
            j = see[i].nonzero()[:, 0]
            x, y = k[j, g], v[j, g]
            qq = q[i, h].to(F64)
            z, size = x @ qq * scale, float((x.abs() @ qq.abs()).max()) * scale
            pr = torch.softmax(z, 0)
            o, a = pr @ y, pr @ y.abs()
            rel = U[F16] + 2 * (2 * (2 * D + 8) * EPS32 * size) + (keys + 16) * 2 * EPS32
            out[i, h] = o
            tol[i, h] = a * rel * 1.01 + U[q.dtype] * 1.001 * o.abs() + SMALL[q.dtype] + \
                len(j) * 2.0 ** -25 * float((pr * s[j, g]).max()) * QMAX[p.type]
    return out, tol


class ScaledPages(Pages):
    def values_of_scales(self, n):
        slot = torch.arange(n)
        return self.host["v_scales"][self.table[0][slot // self.page].long(), slot % self.page].to(F64).abs()

    def scale_v(self, slots, factor):
        for s in slots:
            self.host["v_scales"][int(self.table[0, s // self.page]), s % self.page] *= factor
        self.dev["v_scales"].copy_(self.host["v_scales"])


def chain(n, ctx):
    return torch.cat([torch.ones(n, ctx, dtype=torch.bool), torch.ones(n, n).tril().bool()], 1)


KIND = [(F16, I8), (BF16, I8), (F16, E4M3), (BF16, E4M3)]
ROWS = [(3, 1, 64), (3, 2, 256), (12, 2, 128), (70, 2, 128), (40, 1, 64), (36, 1, 256)]    # tokens, group, head size


@pytest.mark.parametrize("power", [10, 20, 26, 60, 100])
@pytest.mark.parametrize("n,group,dim", ROWS)
@pytest.mark.parametrize("dtype,cache", KIND)
@pytest.mark.parametrize("tree", [False, True])
def test_hidden_finite_scale(tree, dtype, cache, n, group, dim, power):
    """The last token's values are far larger: the rows before it (and its siblings in the tree) give the same bits as
    without, and their own result."""
    g = gen(81 + n + power)
    ctx = 30
    p = ScaledPages(g, [n], [ctx], 1, dim, cache, 16)
    q = (2 * randn(g, n, group, dim)).to(dtype)
    if tree:
        t = random_tree(g, [n])
        t[:, n - 1] = False
        t[n - 1, n - 1] = True
        see = torch.cat([torch.ones(n, ctx, dtype=torch.bool), t], 1)
    else:
        t, see = None, chain(n, ctx)
    want, tol = own64(p, q, see, dim ** -0.5)
    before = attend(p, q, t)
    check(before, want, tol, "ordinary scales")
    p.scale_v([ctx + n - 1], 2.0 ** power)
    got = attend(p, q, t)
    check(got[:-1], want[:-1], tol[:-1], f"a hidden scale 2^{power} larger")
    assert torch.equal(got[:-1], before[:-1])
    if dtype is BF16:
        want, tol = own64(p, q, see, dim ** -0.5)
        check(got[-1], want[-1], tol[-1], "the row that sees it")


@pytest.mark.parametrize("power", [10, 26, 60])
@pytest.mark.parametrize("n,group,dim", ROWS)
@pytest.mark.parametrize("dtype,cache", KIND)
def test_seen_with_no_probability(dtype, cache, n, group, dim, power):
    """Two keys of the context lie 2^-200 below the others and have far larger values."""
    g = gen(91 + n + power)
    ctx = 70
    p = ScaledPages(g, [n], [ctx], 1, dim, cache, 8)
    q = randn(g, n, group, dim).to(dtype)
    q[..., 0] = 8.0
    for s in (3, 40):                        # key: a large negative first value
        at = int(p.table[0, s // 8]), s % 8
        codes = torch.zeros(1, dim)
        codes[..., 0] = -QMAX[cache]
        p.host["k"][at] = codes.to(cache)
        p.host["k_scales"][at] = 200 / QMAX[cache] / 8 * math.sqrt(dim)
    for name in ("k", "k_scales"):
        p.dev[name].copy_(p.host[name])
    p.scale_v([3, 40], 2.0 ** power)
    want, tol = own64(p, q, chain(n, ctx), dim ** -0.5)
    check(attend(p, q, None), want, tol, f"improbable values 2^{power} larger")


@pytest.mark.parametrize("n,group,dim", ROWS)
@pytest.mark.parametrize("cache", [I8, E4M3])
def test_scales_from_key_to_key(cache, n, group, dim):
    """Values of any size from key to key, each row's largest elsewhere; scales of zero and below fp32's normal range."""
    g = gen(101 + n)
    ctx = 200
    p = ScaledPages(g, [n], [ctx], 1, dim, cache, 16)
    q = (2 * randn(g, n, group, dim)).to(BF16)
    p.host["v_scales"] *= 2.0 ** torch.randint(-40, 41, p.host["v_scales"].shape, generator=g)
    p.dev["v_scales"].copy_(p.host["v_scales"])
    want, tol = own64(p, q, chain(n, ctx), dim ** -0.5)
    check(attend(p, q, None), want, tol, "mixed scales")
    for value in (2.0 ** -100, 2.0 ** -130, 0.0, 2.0 ** 100):
        p.host["v_scales"].fill_(value)
        p.dev["v_scales"].copy_(p.host["v_scales"])
        want, tol = own64(p, q, chain(n, ctx), dim ** -0.5)
        got = attend(p, q, None)
        # below 2^-126 the product of scale and code alone keeps 2^-149
        check(got, want, tol + (QMAX[cache] * 2.0 ** -148 if value < 2.0 ** -126 else 0), f"scales of {value}")


@pytest.mark.parametrize("cache", [F16, BF16, I8, E4M3])
@pytest.mark.parametrize("n,group,dim", ROWS)
def test_rows_do_not_meet(cache, n, group, dim):
    """A key that only the last row sees, whose logit there lies far above: the other rows' bits stay."""
    g = gen(111 + n)
    dtype = cache if cache in (F16, BF16) else F16
    p = Pages(g, [n], [90], 1, dim, cache, 16)
    q = (2 * randn(g, n, group, dim)).to(dtype)
    before = attend(p, q, None)
    at = int(p.table[0, (89 + n) // 16]), (89 + n) % 16
    p.dev["k"][at] = (20 * q[-1, :1].float()).clamp(-100, 100).to(p.dev["k"].dtype).cuda() if cache is not E4M3 else \
        (20 * q[-1, :1].float()).clamp(-100, 100).to(E4M3).cuda()
    got = attend(p, q, None)
    assert torch.equal(got[:-1], before[:-1]) and not torch.equal(got[-1], before[-1])
