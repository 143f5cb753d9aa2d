"""svdq_tree_attention at the ends of fp32's and fp16's ranges: logits, scales and queries of any finite size."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from strict import check  # noqa: E402
from test_gpu_cache import (BF16, E4M3, EPS32, F16, F64, I8, QMAX, SMALL, U, Pages, _gpu, attend, attention64, gen,  # noqa: E402, F401
                            randn)

KIND = [(F16, F16), (BF16, BF16), (F16, I8), (BF16, I8), (F16, E4M3), (BF16, E4M3)]
ROWS = [(3, 1, 64), (3, 2, 256), (12, 2, 128), (70, 2, 128), (36, 1, 256)]     # tokens, group, head size


def put(p, name, values, scale=1.0):
    """All of a cache's keys or values, exact in its type; scale: of a cache of codes."""
    p.host[name] = values.to(p.type)
    p.dev[name].copy_(p.host[name])
    if p.type in QMAX:
        p.host[name + "_scales"].fill_(scale)
        p.dev[name + "_scales"].fill_(scale)


def mean_of(p, q, chosen):
    """Output and tolerance of rows that share their weight evenly among chosen [tokens, keys]."""
    n, H, D = q.shape
    v = p.values("v", 0, chosen.shape[1])[0]
    w = chosen.to(F64) / chosen.sum(1, keepdim=True)
    o, a = torch.einsum("nk,kgd->ngd", w, v), torch.einsum("nk,kgd->ngd", w, v.abs())
    o, a = (t.repeat_interleave(H // p.heads, 1) for t in (o, a))
    up = U[F16] if p.type in QMAX else U[q.dtype]
    tol = a * 1.01 * (up + (chosen.shape[1] + 16) * 2 * EPS32) + U[q.dtype] * 1.001 * o.abs() + SMALL[q.dtype]
    if p.type in QMAX:                       # the largest product of probability and scale at 1 or above in fp16
        s = p.host["v_scales"].to(F64).max()
        tol = tol + 2.0 ** -25 * s * QMAX[p.type]
    return o, tol


@pytest.mark.parametrize("size", [15, 20, 24, 25, 27, 28, 30, 40, 60, 100])
@pytest.mark.parametrize("n,group,dim", ROWS)
@pytest.mark.parametrize("dtype,cache", KIND)
def test_logits_of_any_size(dtype, cache, n, group, dim, size):
    """Logits of 0, 1, 2 and 3 times 2^size: the weight lies evenly on the keys of the largest that a row sees."""
    g = gen(121 + n + size)
    ctx = 150
    p = Pages(g, [n], [ctx], 1, dim, cache, 16)
    k = torch.zeros(p.pages, 16, 1, dim)
    level = torch.randint(0, 4, (p.pages, 16, 1), generator=g).float()
    k[..., 0] = 8 * level
    put(p, "k", k)
    q = torch.zeros(n, group, dim, dtype=dtype)
    q[..., 0] = 1024.0
    keys = torch.arange(ctx + n)
    mine = level[p.table[0][keys // 16].long(), keys % 16, 0]
    see = keys <= ctx + torch.arange(n)[:, None]
    top = torch.where(see, mine, -1.0).amax(1, keepdim=True)
    want, tol = mean_of(p, q, see & (mine == top))
    check(attend(p, q, None, scale=2.0 ** (size - 13)), want, tol, f"logits of 2^{size}")
    check(attend(p, -q, None, scale=2.0 ** (size - 13)),
          *mean_of(p, q, see & (mine == torch.where(see, mine, 9.0).amin(1, keepdim=True))), f"logits of -2^{size}")


@pytest.mark.parametrize("n,group,dim", ROWS)
@pytest.mark.parametrize("cache", [I8, E4M3])
@pytest.mark.parametrize("power", [-130, -100, 0, 100, 126])
def test_bf16_queries_keep_small_values(power, cache, n, group, dim):
    """Over codes bf16 queries become fp16: values 2^-20 of a row's largest, which meets keys of zero, carry the logits."""
    g = gen(171 + n + power)
    p = Pages(g, [n], [60], 1, dim, cache, 16)
    k = p.host["k"].float()
    k[..., 0] = 0
    put(p, "k", k, 2.0 ** (10 if power < 100 else -90))
    q = randn(g, n, group, dim)
    if power == -130:                        # steps of 2^-133
        q = (8 * q).round() / 8
    else:
        q *= 2.0 ** -20
        q[..., 0] = 1.0
    q = (q * 2.0 ** power).to(BF16)
    # logits of size one or so
    scale = 2.0 ** min(110, max(-110, -power - (7 if cache is I8 else 9) + (20 if power != -130 else 0) - (10 if power < 100 else -90) - 3))
    want, tol = attention64(p, q, None, scale, U[F16])
    check(attend(p, q, None, scale=scale), want, tol, f"queries of 2^{power}")


@pytest.mark.parametrize("n,group,dim", ROWS)
@pytest.mark.parametrize("dtype,cache", KIND)
def test_scales_at_the_ends(dtype, cache, n, group, dim):
    """The largest and smallest scale with queries of zero."""
    g = gen(181 + n)
    p = Pages(g, [n], [60], 1, dim, cache, 16)
    see = torch.arange(60 + n) <= 60 + torch.arange(n)[:, None]
    for scale in (2.0 ** -126, 2.0 ** 126):
        q = torch.zeros(n, group, dim, dtype=dtype)
        check(attend(p, q, None, scale=scale), *mean_of(p, q, see), f"queries of zero, {scale}")


@pytest.mark.parametrize("n,group,dim", ROWS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_far_logits_by_the_largest_scale(dtype, n, group, dim):
    """Logits of 0 to 3 times 2^115 from queries of 2^-14 and a scale of 2^126."""
    g = gen(191 + n)
    p = Pages(g, [n], [150], 1, dim, dtype, 16)
    k = torch.zeros(p.pages, 16, 1, dim)
    level = torch.randint(0, 4, (p.pages, 16, 1), generator=g).float()
    k[..., 0] = 8 * level
    put(p, "k", k)
    q = torch.zeros(n, group, dim, dtype=dtype)
    q[..., 0] = 2.0 ** -14
    keys = torch.arange(150 + n)
    mine = level[p.table[0][keys // 16].long(), keys % 16, 0]
    see = keys <= 150 + torch.arange(n)[:, None]
    top = torch.where(see, mine, -1.0).amax(1, keepdim=True)
    check(attend(p, q, None, scale=2.0 ** 126), *mean_of(p, q, see & (mine == top)), "far logits")
