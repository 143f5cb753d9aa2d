"""The operators of a transformer block between its quantized linears, against plain 64-bit
implementations: svdq_add_rmsnorm, svdq_gemm_act_residual, svdq_rope_axes.

Tolerances are derived: U is half an ulp of the output's type relative to the value, EPS32 the
fp32 rounding unit; sums of n fp32 terms in any order are off by at most n EPS32 of the sum of
the terms' magnitudes (2 EPS32 per term for the matrix cores, whose partial sums may truncate).
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_w4a4_quantized_amd import binding  # noqa: E402

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
E4M3 = torch.float8_e4m3fn
EPS32 = 2.0 ** -24
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
SMALL = {F16: 2.0 ** -25, BF16: 2.0 ** -134}       # half the smallest step
TINY = 2.0 ** -100


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.lib()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


def guarded(rows, cols, dtype, pad=0):
    """A device view [rows, cols] inside a buffer of 72s, to see writes outside it."""
    step = cols + pad
    buf = torch.full((2 + rows, step), 72, dtype=dtype, device="cuda") if dtype is torch.int8 else \
        torch.full((2 + rows, step), 72.0, device="cuda").to(dtype)
    return buf, buf[1:1 + rows, :cols]


def untouched(buf, rows, cols):
    f = buf.float().cpu()
    return bool((f[0] == 72).all() and (f[1 + rows:] == 72).all() and (f[1:1 + rows, cols:] == 72).all())


def check(got, want, tol, what):
    got, want = got.to(F64).cpu(), want.to(F64).cpu()
    assert got.shape == want.shape, what
    bad = (got - want).abs() > tol
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst " \
        f"{float((got - want).abs().max())} at tolerance {float(torch.as_tensor(tol).max())}"


# ------------------------------------------------------------------ norm
def norm64(x, residual, w, eps, out_format, K):
    h, stream = x.to(F64), None
    if residual is not None:
        stream = (x.float() + residual.float()).to(residual.dtype)
        h = stream.to(F64)
    rstd = 1 / torch.sqrt((h * h).sum(-1) / K + eps)
    v = h * w.to(F64)
    if out_format == "same":
        return v * rstd[:, None], None, stream
    qmax = 127.0 if out_format == "int8" else 448.0
    a = v.abs().amax(-1).clamp_min(TINY)
    return v * (qmax / a)[:, None], a * rstd / qmax, stream


def codes32(x, residual, w, out_format):
    """The codes by fp32 elementwise operations, as the definition states them."""
    h = x.float().numpy()
    if residual is not None:
        h = (x.float() + residual.float()).to(residual.dtype).float().numpy()
    v = h * w.float().numpy()
    a = np.maximum(np.abs(v).max(-1, keepdims=True), np.float32(TINY))
    q = v * (np.float32(127.0 if out_format == "int8" else 448.0) / a)
    return torch.from_numpy(np.rint(q)).to(torch.int8) if out_format == "int8" else torch.from_numpy(q).to(E4M3)


def norm_case(M, K, xt, rt, wt, out_format, pad, seed, x_scale=1.0):
    g = gen(seed)
    xb = (randn(g, M, K + pad) * x_scale).to(xt)
    x = xb[:, :K]
    r = None if rt is None else (randn(g, M, K) * 3 * x_scale).to(rt)
    w = (1 + 0.2 * randn(g, K)).to(wt)
    eps = 1e-6
    xd = xb.cuda()[:, :K]
    ob, out = guarded(M, K, {"int8": torch.int8, "e4m3": E4M3, "same": xt}[out_format])
    sb, ro = (None, None) if r is None else guarded(M, K, rt, pad)
    y, s, st = binding.svdq_add_rmsnorm(xd, w.cuda(), eps, residual=None if r is None else r.cuda(),
                                        out_format=out_format, out=out, residual_out=ro)
    torch.cuda.synchronize()
    assert untouched(ob, M, K)
    want, sw, stream = norm64(x, r, w, eps, out_format, K)
    if r is not None:
        assert untouched(sb, M, K)
        assert torch.equal(st.cpu(), stream)
    tol32 = (K / 64 + 16) * EPS32            # the row sum's lanes and steps, the root, the products
    if out_format == "same":
        assert s is None
        check(y, want, (U[xt] * 1.001 + tol32) * want.abs() + SMALL[xt], "out")
    else:
        check(s, sw, sw * tol32, "scales")
        assert torch.equal(y.cpu().view(torch.uint8), codes32(x, r, w, out_format).view(torch.uint8))
        step = 0.5 if out_format == "int8" else torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10))
        check(y, want, step + want.abs() * 3 * EPS32, "codes")


@pytest.mark.parametrize("out_format", ["int8", "e4m3", "same"])
@pytest.mark.parametrize("xt,rt,wt", [(F16, None, F32), (BF16, BF16, BF16), (F16, F32, F16), (BF16, F32, F32),
                                      (F16, F16, F32)])
@pytest.mark.parametrize("M,K,pad", [(1, 1, 0), (3, 7, 0), (1, 3072, 0), (5, 1111, 3), (129, 256, 8), (4, 4097, 0),
                                     (7, 4096, 5)])
def test_norm(M, K, pad, xt, rt, wt, out_format):
    norm_case(M, K, xt, rt, wt, out_format, pad, M * 131 + K)


@pytest.mark.parametrize("K", [8, 512, 1000, 1024, 1032, 2048, 3000, 5000, 8192, 8200, 12288, 16384, 16392, 40003])
@pytest.mark.parametrize("out_format", ["int8", "same"])
def test_norm_widths(K, out_format):
    norm_case(3, K, BF16, F32, F32, out_format, 0, K)
    norm_case(2, K, F16, F16, F16, out_format, 1, K + 1)


@pytest.mark.parametrize("M", [2, 4, 31, 257, 1030, 5000])
def test_norm_rows(M):
    norm_case(M, 320, BF16, BF16, F32, "int8", 0, M)
    norm_case(M, 2056, F16, None, F32, "e4m3", 0, M + 1)


def test_norm_extremes():
    """Rows of zeros, rows far below and above one, a single large value: finite scales, exact codes."""
    for xt, scales in ((BF16, (0.0, 1e-30, 1e-12, 1e15)), (F16, (0.0, 2e-7, 1e-3, 200.0))):
        for scale in scales:
            for out_format in ("int8", "e4m3", "same"):
                norm_case(4, 200, xt, xt, F32, out_format, 0, 5, scale)
    x = torch.zeros(2, 4096, dtype=BF16)
    x[0, 4095], x[1, 0] = -3e4, 1e-3
    y, s, _ = binding.svdq_add_rmsnorm(x.cuda(), torch.ones(4096).cuda(), 1e-6)
    y, s = y.cpu(), s.cpu()
    assert int(y[0, 4095]) == -127 and int(y[1, 0]) == 127 and int((y != 0).sum()) == 2
    assert bool(torch.isfinite(s).all())


@pytest.mark.parametrize("K", [700, 40000])
@pytest.mark.parametrize("rt", [None, BF16, F32])
@pytest.mark.parametrize("out_format", ["int8", "e4m3", "same"])
def test_norm_not_finite(out_format, rt, K):
    """An infinity or NaN shows in its own row's scale (or value) and in no other row."""
    g = gen(11)
    x, w = randn(g, 6, K).to(BF16), 1 + 0.2 * randn(g, K)
    r = None if rt is None else randn(g, 6, K).to(rt).cuda()
    clean = binding.svdq_add_rmsnorm(x.cuda(), w.cuda(), residual=r, out_format=out_format)
    bad = [(1, 3, math.inf), (2, K - 1, math.nan), (4, 0, -math.inf)]
    for row, col, v in bad:
        x[row, col] = v
    got = binding.svdq_add_rmsnorm(x.cuda(), w.cuda(), residual=r, out_format=out_format)
    rows = [0, 3, 5]
    for a, b in zip(clean, got):
        if a is not None:
            assert torch.equal(a.cpu()[rows].contiguous().view(torch.uint8), b.cpu()[rows].contiguous().view(torch.uint8))
    for row, col, _ in bad:
        assert math.isnan(float(got[0][row, col] if out_format == "same" else got[1][row]))


def test_norm_in_place_and_streams():
    """The stream written over the residual, and over x; work on a side stream given by its handle."""
    g = gen(3)
    x, r, w = randn(g, 65, 3072).to(BF16), randn(g, 65, 3072).to(BF16), torch.ones(3072)
    a = binding.svdq_add_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda())
    rc = r.cuda()
    b = binding.svdq_add_rmsnorm(x.cuda(), w.cuda(), residual=rc, residual_out=rc)
    assert b[2] is rc and all(torch.equal(p, q) for p, q in zip(a, b))
    xc = x.cuda()
    b = binding.svdq_add_rmsnorm(xc, w.cuda(), residual=r.cuda(), residual_out=xc)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    side = torch.cuda.Stream()
    xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
    side.wait_stream(torch.cuda.current_stream())
    c = binding.svdq_add_rmsnorm(xd, wd, residual=rd, stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, c))


# ------------------------------------------------------------------ product
def act64(v, act):
    if act == "gelu":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v * torch.sigmoid(v) if act == "silu" else v


def gemm_case(M, N, K, t, out=F16, act="none", bias=True, residual=True, scales=True, xpad=0, ypad=0, seed=0,
              inplace=False):
    g = gen(seed + M + 7 * N + 13 * K)
    if t is torch.int8:
        xb = torch.randint(-127, 128, (M, K + xpad), generator=g).to(t)
        w = torch.randint(-127, 128, (N, K), generator=g).to(t)
        norm = 1 / (73.0 * 73.0 * math.sqrt(K))
    else:
        xb = randn(g, M, K + xpad).to(t)
        w = randn(g, N, K).to(t)
        norm = 1 / math.sqrt(K)
    xs = (0.5 + torch.rand(M, generator=g)) * math.sqrt(norm) if scales else None
    ws = (0.5 + torch.rand(N, generator=g)) * math.sqrt(norm) if scales else None
    b = randn(g, N).to(out) if bias else None
    r = randn(g, M, N).to(out) if residual else None
    x = xb[:, :K]
    buf, y = guarded(M, N, out, ypad)
    if inplace:
        y.copy_(r)
        rd = y
    else:
        rd = None if r is None else r.cuda()
    dev = lambda v: None if v is None else v.cuda()  # noqa: E731
    binding.svdq_gemm_act_residual(xb.cuda()[:, :K], w.cuda(), dev(xs), dev(ws), dev(b), act, rd, out, y)
    torch.cuda.synchronize()
    assert untouched(buf, M, N)
    X, W = x.to(F64), w.to(F64)
    acc, mag = X @ W.T, X.abs() @ W.abs().T
    # FP8 matrix cores align eight products to the largest with 13 bits below it and drop the rest
    # of the other seven: found with one large product beside small ones, not with this test's data
    eights = 7 * 2.0 ** -13 * mag if t is E4M3 else 0
    sum_tol = eights + (0 if t is torch.int8 else 2 * K * EPS32) * mag + EPS32 * acc.abs()
    s = 1.0 if not scales else xs.to(F64)[:, None] * ws.to(F64)
    v = acc * s
    tol = sum_tol * s + 3 * EPS32 * v.abs()
    if bias:
        v = v + b.to(F64)
        tol = tol + EPS32 * v.abs()
    # the activations' slopes are at most 1.13; their fp32 forms are within 2^-19 of the value and
    # lose nothing else: exp and reciprocal are good to an ulp of arguments of a few dozen
    z = act64(v, act)
    if act != "none":
        tol = 1.13 * tol + 2.0 ** -19 * v.abs()
    if residual:
        z = z + r.to(F64)
    check(y, z, tol + (U[out] * 1.001 + EPS32) * z.abs() + U[out] * tol + SMALL[out], f"y {M}x{N}x{K} {t} {act}")


TYPES = [torch.int8, E4M3, F16, BF16]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 64, 128), (2, 17, 48), (3, 130, 1040), (17, 48, 4096), (33, 129, 80),
                                   (64, 256, 512), (65, 100, 144), (128, 128, 256), (129, 257, 272), (200, 1000, 1008)])
def test_gemm(M, N, K, t):
    out = F16 if (M + N) % 2 else BF16
    gemm_case(M, N, K, t, out, act=("none", "gelu", "silu")[(M + N + K) % 3], scales=t in (torch.int8, E4M3) or K == 80)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("bias,residual,scales", [(False, False, False), (True, False, True), (False, True, True)])
def test_gemm_epilogue(t, act, bias, residual, scales):
    for out in (F16, BF16):
        gemm_case(70, 136, 192, t, out, act, bias, residual, scales or t is torch.int8)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,N,K,xpad,ypad", [(40, 72, 160, 16, 8), (40, 72, 160, 48, 3), (5, 33, 64, 32, 1),
                                             (300, 520, 384, 16, 8)])
def test_gemm_strides(t, M, N, K, xpad, ypad):
    gemm_case(M, N, K, t, BF16, "silu", xpad=xpad, ypad=ypad)
    gemm_case(M, N, K, t, F16, "none", xpad=xpad, ypad=ypad, inplace=True)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,N,K", [(600, 1100, 1040), (1000, 2304, 2064), (1537, 3000, 640), (2100, 2060, 128)])
def test_gemm_many_tiles(t, M, N, K):
    gemm_case(M, N, K, t, F16, "gelu")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,N,K,ypad", [(500, 9201, 2064, 0), (770, 9210, 2064, 6), (1000, 3075, 4112, 5)])
def test_gemm_wide_tiles(t, M, N, K, ypad):
    gemm_case(M, N, K, t, BF16, "silu", ypad=ypad)


@pytest.mark.parametrize("M", [1, 2, 5, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 128, 160])
def test_gemm_few_rows(M):
    gemm_case(M, 528, 3072, TYPES[M % 4], BF16, "silu", scales=True)
    gemm_case(M, 96, 4112, TYPES[(M + 1) % 4], F16, "none", scales=True)


@pytest.mark.parametrize("t", [E4M3, F16, BF16])
@pytest.mark.parametrize("M", [5, 70, 300, 2500])
def test_gemm_not_finite(t, M):
    """NaN behind the rows of x reaches nothing; in x, w or the residual its own row, column or element."""
    g = gen(12 + M)
    N, K = 2060, 208
    xb, w, r = randn(g, M, K + 16).to(t), randn(g, N, K).to(t), randn(g, M, N).to(F16)
    clean = binding.svdq_gemm_act_residual(xb.cuda()[:, :K], w.cuda(), residual=r.cuda(), out_dtype=F16).cpu()
    assert bool(torch.isfinite(clean).all())
    xb[:, K:] = math.nan
    xb[2, K - 1] = math.nan
    w[N - 1, 0] = math.nan
    r[0, 1] = math.nan
    got = binding.svdq_gemm_act_residual(xb.cuda()[:, :K], w.cuda(), residual=r.cuda(), out_dtype=F16).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[2], want[:, N - 1], want[0, 1] = True, True, True
    assert torch.equal(torch.isnan(got), want)
    assert torch.equal(got[~want], clean[~want])


def test_gemm_int8_sums_are_exact():
    """The largest codes at a long K: fp32 sums would lose the last bits of 127 * 127 * K."""
    K = 1 << 17
    x = torch.full((3, K), 127, dtype=torch.int8)
    x[1] = -127
    x[2, ::2] = -127
    w = torch.full((5, K), 127, dtype=torch.int8)
    w[3, -1] = 126                           # one step less in one product
    s = torch.tensor([2.0 ** -20] * 3).cuda()
    y = binding.svdq_gemm_act_residual(x.cuda(), w.cuda(), xs=s, out_dtype=F16).cpu().to(F64)
    want = (x.to(F64) @ w.to(F64).T) * 2.0 ** -20
    assert torch.equal(y, want.to(F16).to(F64))
    x = torch.zeros((1, K), dtype=torch.int8)
    x[0, -1], x[0, 0] = 1, 1
    assert float(binding.svdq_gemm_act_residual(x.cuda(), w.cuda())[0, 3]) == 253.0


def test_gemm_e4m3_sums():
    """Products that share a binary order lose nothing: 8 ... 15 times 8 ... 15, signs mixed, and
    every product counts (each value of K alone)."""
    g = gen(5)
    x = (torch.randint(8, 16, (70, 1040), generator=g) * (torch.randint(0, 2, (70, 1040), generator=g) * 2 - 1)).float()
    w = (torch.randint(8, 16, (90, 1040), generator=g) * (torch.randint(0, 2, (90, 1040), generator=g) * 2 - 1)).float()
    s = torch.full((70,), 2.0 ** -4).cuda()
    for M in (3, 70):
        y = binding.svdq_gemm_act_residual(x[:M].to(E4M3).cuda(), w.to(E4M3).cuda(), xs=s[:M], out_dtype=F16).cpu()
        assert torch.equal(y, (x[:M].to(F64) @ w.to(F64).T * 2.0 ** -4).to(F16))
    one = torch.eye(272).to(E4M3).cuda()
    y = binding.svdq_gemm_act_residual(one, one, out_dtype=F16).cpu()
    assert torch.equal(y, torch.eye(272, dtype=F16))


def test_gemm_same_bits_and_empty():
    g = gen(9)
    for t, M in ((torch.int8, 300), (BF16, 300), (E4M3, 3), (F16, 40)):
        x, w = randn(g, M, 1024).to(t).cuda(), randn(g, 640, 1024).to(t).cuda()
        y = [binding.svdq_gemm_act_residual(x, w, out_dtype=BF16) for _ in range(3)]
        assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
    assert binding.svdq_gemm_act_residual(x[:0], w).shape == (0, 640)
    assert binding.svdq_gemm_act_residual(x, w[:0]).shape == (40, 0)


# ------------------------------------------------------------------ rotary positions
def rope64(x, w, positions, inv_freq, axis_pairs, pairs, eps, inverse):
    u = x.to(F64)
    if w is not None:
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps) * w.to(F64)
    axis = sum(([i] * n for i, n in enumerate(axis_pairs)), [])
    angle = positions.to(F64)[..., axis] * inv_freq.to(F64)     # [(batch,) tokens, pairs]
    c, s = torch.cos(angle).unsqueeze(-2), torch.sin(angle).unsqueeze(-2)
    s = -s if inverse else s
    P = len(axis)
    i = torch.arange(P) * 2 if pairs == "adjacent" else torch.arange(P)
    j = i + 1 if pairs == "adjacent" else i + P
    y = u.clone()
    y[..., i] = u[..., i] * c - u[..., j] * s
    y[..., j] = u[..., i] * s + u[..., j] * c
    size = u.abs()
    size[..., i] = size[..., j] = torch.maximum(u[..., i].abs(), u[..., j].abs())
    return y, size


def rope_inputs(B, T, H, G, D, axis_pairs, dtype, seed, far=1):
    g = gen(seed)
    qkv = randn(g, B, T, (H + 2 * G) * D).to(dtype)
    q, k = qkv[..., :H * D].unflatten(-1, (H, D)), qkv[..., H * D:(H + G) * D].unflatten(-1, (G, D))
    pos = torch.randint(0, 200 * far, (T, len(axis_pairs)), generator=g, dtype=torch.int32)
    freq = torch.cat([10000.0 ** (-torch.arange(n, dtype=F64) / max(n, 1)) for n in axis_pairs]).float()
    return g, qkv, q, k, pos, freq


def rope_case(B, T, H, G, D, axis_pairs, pairs="adjacent", dtype=F16, norm=True, inverse=False, heads_first=False,
              far=1, seed=0, batch_positions=False, fp32_positions=False):
    g, qkv, q, k, pos, freq = rope_inputs(B, T, H, G, D, axis_pairs, dtype, seed + T + D, far)
    if batch_positions:
        pos = torch.stack([pos + b for b in range(B)])
    if fp32_positions:
        pos = pos.float() + 0.25
    qw, kw = ((1 + 0.2 * randn(g, D)), (1 + 0.2 * randn(g, D))) if norm else (None, None)
    dev = qkv.cuda()
    qd, kd = dev[..., :H * D].unflatten(-1, (H, D)), dev[..., H * D:(H + G) * D].unflatten(-1, (G, D))
    cu = lambda v: None if v is None else v.cuda()  # noqa: E731
    got = binding.svdq_rope_axes(qd, kd, pos.cuda(), freq.cuda(), axis_pairs, pairs, cu(qw), cu(kw), 1e-6, inverse,
                                 heads_first)
    torch.cuda.synchronize()
    assert torch.equal(dev.cpu(), qkv)       # the packed projection is only read
    for x, w, y in ((q, qw, got[0]), (k, kw, got[1])):
        want, size = rope64(x, w, pos, freq, axis_pairs, pairs, 1e-6, inverse)
        y = y.transpose(1, 2) if heads_first else y
        # cosines and sines within 2^-21, the norm's sum and root, one rounding
        tol = (U[dtype] * 1.001) * want.abs() + (2.0 ** -20 + (D / 8 + 8) * EPS32) * size + SMALL[dtype]
        check(y, want, tol, f"rope {B}x{T}x{H}/{G}x{D} {pairs}")


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("dtype,norm", [(F16, True), (BF16, False), (BF16, True), (F16, False)])
@pytest.mark.parametrize("D,axis_pairs", [(128, (8, 28, 28)), (64, (32,)), (128, (16, 16)), (80, (10, 14, 16)),
                                          (72, (12, 12, 12)), (256, (40, 44, 44)), (2, (1,)), (6, (1, 1, 1)),
                                          (10, (3,)), (96, (0, 24)), (130, (1, 2, 3, 4)), (7, (2,)), (1024, (512,))])
def test_rope(D, axis_pairs, dtype, norm, pairs):
    rope_case(1, 5, 3, 2, D, axis_pairs, pairs, dtype, norm)
    rope_case(2, 3, 4, 1, D, axis_pairs, pairs, dtype, norm, heads_first=True, batch_positions=True)


@pytest.mark.parametrize("T,H,G", [(1, 24, 24), (1, 1, 1), (2, 32, 8), (63, 24, 24), (64, 40, 8), (65, 5, 1),
                                   (1000, 24, 24), (4097, 8, 2)])
def test_rope_tokens(T, H, G):
    rope_case(1, T, H, G, 128, (8, 28, 28))
    rope_case(1, T, H, G, 128, (16, 24, 24), "halves", BF16, False, heads_first=True)


def test_rope_many_tokens():
    rope_case(2, 9000, 8, 2, 64, (4, 14, 14), "adjacent", BF16, True, heads_first=True)


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("B,T,H,G,D", [(1, 5500, 2, 1, 256), (3, 3000, 1, 1, 64), (1, 4100, 3, 1, 128), (2, 2100, 5, 3, 8),
                                       (2500, 3, 7, 1, 64), (1, 6150, 6, 2, 16)])
def test_rope_tokens_of_few_heads(B, T, H, G, D, heads_first):
    """A wave takes several tokens, across batches too: one head, odd heads, few tokens a batch."""
    rope_case(B, T, H, G, D, (D // 2,), "adjacent", BF16, True, heads_first=heads_first)


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("D", [128, 36])
def test_rope_far_positions(D, pairs):
    """Positions up to 2,000,000: an fp32 product alone would be off by 0.06 radians."""
    rope_case(1, 300, 2, 1, D, (D // 2,), pairs, F16, False, far=10000)


def test_rope_positions_kinds():
    rope_case(3, 20, 4, 2, 128, (8, 28, 28), batch_positions=True, fp32_positions=True)
    rope_case(3, 20, 4, 2, 128, (8, 28, 28), "halves", fp32_positions=True)
    g, qkv, q, k, pos, freq = rope_inputs(1, 40, 4, 2, 128, (64,), F16, 2)
    both = binding.svdq_rope_axes(q.cuda(), k.cuda(), pos.cuda(), freq.cuda(), (64,))
    one, none = binding.svdq_rope_axes(q[0].cuda(), None, pos.cuda(), freq.cuda(), (64,))   # no batch, no keys
    assert none is None and torch.equal(one, both[0][0])
    zero = binding.svdq_rope_axes(q.cuda(), k.cuda(), (-pos).cuda(), freq.cuda(), (64,))    # negative positions
    back = binding.svdq_rope_axes(q.cuda(), k.cuda(), pos.cuda(), freq.cuda(), (64,), inverse=True)
    assert torch.equal(zero[0], back[0]) and torch.equal(zero[1], back[1])


@pytest.mark.parametrize("D,axis_pairs", [(128, (8, 28, 28)), (80, (10, 20)), (6, (2,))])
@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_rope_in_place(D, axis_pairs, pairs):
    g, qkv, q, k, pos, freq = rope_inputs(2, 37, 6, 2, D, axis_pairs, BF16, 4)
    w = (1 + 0.2 * randn(g, D)).cuda()
    a = binding.svdq_rope_axes(q.cuda(), k.cuda(), pos.cuda(), freq.cuda(), axis_pairs, pairs, w, w)
    dev = qkv.cuda()
    qd, kd = dev[..., :6 * D].unflatten(-1, (6, D)), dev[..., 6 * D:8 * D].unflatten(-1, (2, D))
    binding.svdq_rope_axes(qd, kd, pos.cuda(), freq.cuda(), axis_pairs, pairs, w, w, q_out=qd, k_out=kd)
    assert torch.equal(qd, a[0]) and torch.equal(kd, a[1])
    assert torch.equal(dev[..., 8 * D:].cpu(), qkv[..., 8 * D:])      # the values behind them are untouched


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("D,axis_pairs", [(128, (8, 28, 28)), (20, (3, 5))])
def test_rope_gradient(D, axis_pairs, pairs):
    """inverse is the gradient: against autograd of the 64-bit formula, and against differences."""
    rope_case(2, 11, 4, 2, D, axis_pairs, pairs, F16, False, inverse=True)
    g, qkv, q, k, pos, freq = rope_inputs(1, 7, 3, 1, D, axis_pairs, F16, 6)
    up = randn(g, *q.shape).to(F16)
    x = q.to(F64).requires_grad_()
    y, _ = rope64(x, None, pos, freq, axis_pairs, pairs, 1e-6, False)
    (y * up.to(F64)).sum().backward()
    run = lambda v, inv: binding.svdq_rope_axes(v.cuda(), None, pos.cuda(), freq.cuda(), axis_pairs, pairs,  # noqa: E731
                                                inverse=inv)[0].cpu().to(F64)
    grad = run(up, True)
    _, size = rope64(up, None, pos, freq, axis_pairs, pairs, 1e-6, True)
    check(grad, x.grad, U[F16] * 1.001 * x.grad.abs() + 2.0 ** -20 * size + SMALL[F16], "gradient")
    # the map is linear, so a difference over a whole step of 2 along d is exact but for roundings
    d = randn(g, *q.shape).to(F16).sign()
    hi, lo = (q + d).to(F16), (q - d).to(F16)
    yh, yl = run(hi, False), run(lo, False)
    num = ((yh - yl) / 2 * up.to(F64)).sum()
    ana = (grad * (hi.to(F64) - lo.to(F64)) / 2).sum()
    tol = (up.to(F64).abs() * (U[F16] + 2.0 ** -19) * (yh.abs() + yl.abs() + 4)).sum() + \
        ((U[F16] + 2.0 ** -19) * (grad.abs() + size) * (hi.to(F64) - lo.to(F64)).abs()).sum()
    assert abs(float(num - ana)) <= float(tol)


# ------------------------------------------------------------------ graphs
def test_operators_in_a_graph():
    """Norm, product and positions captured on a side stream and replayed with new inputs."""
    g = gen(11)
    K, N, T = 256, 3 * 256, 96
    x, r, w = randn(g, T, K).to(BF16).cuda(), randn(g, T, K).to(BF16).cuda(), torch.ones(K).cuda()
    wq = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8).cuda()
    ws = (torch.rand(N, generator=g) / 2000).cuda()
    pos = torch.arange(T, dtype=torch.int32).unsqueeze(-1).cuda()
    freq = (10000.0 ** (-torch.arange(32) / 32)).cuda()

    def block():
        c, s, h = binding.svdq_add_rmsnorm(x, w, residual=r)
        y = binding.svdq_gemm_act_residual(c, wq, s, ws, out_dtype=BF16)
        q, k = y[:, :K].unflatten(-1, (4, 64)), y[:, K:2 * K].unflatten(-1, (4, 64))
        return (h, *binding.svdq_rope_axes(q, k, pos, freq, (32,)))

    block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    for i in range(5):
        x.copy_(randn(g, T, K).to(BF16))
        want = [t.clone() for t in block()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_gemm_workspace():
    """Splits of K need the workspace they ask for; less is allowed and never written past; INT8
    sums do not depend on it."""
    g = gen(13)
    M, N, K = 70, 200, 8192
    need = binding.gemm_act_residual_workspace_bytes(M, N, K, 3)
    assert need > 0
    x = torch.randint(-127, 128, (M, K), generator=g).to(torch.int8).cuda()
    w = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8).cuda()
    s = torch.full((M,), 2.0 ** -16).cuda()
    want = (x.cpu().to(F64) @ w.cpu().to(F64).T * 2.0 ** -16).to(F16)
    for room in (need, need // 2 // 16 * 16, 16, 0):
        buf = torch.full((room + 64,), 77, dtype=torch.uint8, device="cuda")
        y = binding.svdq_gemm_act_residual(x, w, xs=s, workspace=buf[:room])
        assert torch.equal(y.cpu(), want) and bool((buf[room:] == 77).all())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,N,K", [(65, 64, 8192), (100, 300, 5008), (130, 520, 4096), (70, 3072, 4096), (16, 48, 12288),
                                   (64, 100, 8192)])
def test_gemm_splits(t, M, N, K):
    gemm_case(M, N, K, t, BF16, "gelu", scales=True)
