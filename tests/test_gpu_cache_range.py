"""svdq_tree_attention at the ends of fp32's and fp16's ranges: logits, scales and queries of any finite size."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from strict import check  # noqa: E402
from test_gpu_cache import (BF16, E4M3, EPS32, F16, F64, I8, QMAX, SMALL, U, Pages, _gpu, attend, gen,  # noqa: E402, F401
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
