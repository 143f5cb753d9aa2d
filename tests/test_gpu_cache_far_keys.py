"""svdq_tree_attention where one key lies far above very many others that carry the whole output: what is small next to a
row's largest probability still counts.

A probability (with an 8-bit cache its product with V's scale) is an fp16 operand relative to the row's largest, which
lies at 2^7 or above: below fp16's normal range it is off by 2^-25 of one, 2^-32 of the largest; bf16 keeps its 8 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from strict import check  # noqa: E402
from test_gpu_cache import BF16, E4M3, EPS32, F16, F64, I8, QMAX, SMALL, U, Pages, _gpu, attend, gen  # noqa: E402, F401
from test_gpu_cache_range import put  # noqa: E402

CTX = 131070


@pytest.mark.parametrize("n,group,dim", [(1, 1, 64), (3, 2, 128), (12, 2, 64), (40, 1, 64), (40, 1, 128)])    # tokens, group, head size
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (F16, I8), (BF16, E4M3)])
def test_many_keys_far_below(dtype, cache, n, group, dim):
    g = gen(131 + n)
    p = Pages(g, [n], [CTX], 1, dim, cache, 64, spare=0)
    code = QMAX.get(cache, 1.0)              # of a value of one
    column = torch.where(torch.arange(dim) % 2 == 0, 1.0, 0.5)
    for at, nats in ((0, 18.0), (70001, 18.0), (CTX - 1, 18.0), (333, 20.0)):
        k, v = torch.zeros(p.pages, 64, 1, dim), (code * column).expand(p.pages, 64, 1, dim).clone()
        where = int(p.table[0, at // 64]), at % 64
        k[where][..., 0] = 8.0
        v[where] = 0.0
        put(p, "k", k)
        put(p, "v", v, 1.0 / code)
        q = torch.zeros(n, group, dim, dtype=dtype)
        q[..., 0] = nats
        far = (CTX + torch.arange(n, dtype=F64))[:, None, None] * math.exp(-nats)
        want = (far / (1 + far) * column.to(F64) if cache is not E4M3 else far / (1 + far) * (code * column).to(E4M3).to(F64) / code)
        want = want.expand(n, group, dim)
        keys = CTX + n
        up = U[F16] if cache in QMAX else U[dtype]
        tol = want * (up + keys * 2 * EPS32 + 100 * EPS32 * nats) + U[dtype] * 1.001 * want + SMALL[dtype]
        if dtype is F16 or cache in QMAX:
            tol = tol + keys * 2.0 ** -32
        check(attend(p, q, None, scale=0.125), want, tol, f"{nats} nats below key {at}")
        # all keys in one part
        one = attend(p, q, None, scale=0.125, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
        check(one, want, tol, f"{nats} nats below key {at}, undivided")
