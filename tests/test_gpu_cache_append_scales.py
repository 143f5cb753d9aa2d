"""Codes and scales of svdq_rope_append bit for bit where nothing is rounded before: values, and keys at position 0."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_w4a4_quantized_amd import binding  # noqa: E402
from test_gpu_cache import BF16, E4M3, F16, I8, QMAX, Pages, _gpu, gen, randn, raw  # noqa: E402, F401


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 256])
@pytest.mark.parametrize("dtype,cache", [(F16, I8), (BF16, I8), (F16, E4M3), (BF16, E4M3)])
def test_scales_are_quotients(dtype, cache, dim, odd):
    """a / qmax and rnd(u (qmax / a)) in fp32; odd: the step's tokens at addresses that the wide kernel does not take."""
    g = gen(161 + dim)
    n, kv, page = 300, 3, 16
    p = Pages(g, [n], [5], kv, dim, cache, page)
    rows = (randn(g, n, 2 * kv * dim + odd) * 2.0 ** torch.randint(-8, 6, (n, 1), generator=g)).to(dtype)
    k, v = (t.unflatten(-1, (kv, dim)) for t in rows[:, odd:].split([kv * dim, kv * dim], -1))
    dev = rows.cuda()
    kd, vd = (t.unflatten(-1, (kv, dim)) for t in dev[:, odd:].split([kv * dim, kv * dim], -1))
    freq = torch.full((dim // 2,), 0.3, device="cuda")
    binding.svdq_rope_append(p.cache, p.batch, None, kd, vd, torch.zeros(n, 1, dtype=torch.int32, device="cuda"), freq, (dim // 2,))
    slot = 5 + torch.arange(n)
    at = p.table[0][slot // page].long(), slot % page
    for name, x in (("k", k.float()), ("v", v.float())):
        a = x.abs().amax(-1).clamp_min(2.0 ** -100)
        qmax = torch.full_like(a, QMAX[cache])
        assert torch.equal(p.dev[name + "_scales"].cpu()[at], a / qmax)
        codes = x * (qmax / a)[..., None]
        codes = codes.round().to(I8) if cache is I8 else codes.to(E4M3)
        assert torch.equal(raw(p.dev[name]).cpu()[at], raw(codes))
