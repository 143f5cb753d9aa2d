"""The block operators at the edges of their definitions: sums of products of very different sizes,
and whatever else an ordinary input does not show.  Exact where the definition is."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_w4a4_quantized_amd import binding  # noqa: E402
from test_gpu_block import EPS32, SMALL, U, check, norm64, norm_case, rope64  # noqa: E402

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.lib()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("out_format", ["int8", "e4m3", "same"])
@pytest.mark.parametrize("rt", [None, BF16, F32])
@pytest.mark.parametrize("K", [1, 200, 1500, 2000, 5000, 12288, 30000, 40003])
def test_norm_of_large_values(K, rt, out_format):
    """Values whose squares, or the sum of them, pass fp32's range (from 1.8e19 on), beside ordinary
    rows of the same workgroup: the tolerances of every other row."""
    scale = torch.tensor([1.0, 1e18, 1e19, 1e25, 3.0, 1e33, 1e37, 0.0, 1e37])[:, None]
    norm_case(9, K, BF16, rt, F32, out_format, 0, K, scale)


@pytest.mark.parametrize("out_format", ["int8", "same"])
@pytest.mark.parametrize("K", [700, 2000, 5000, 40000])
def test_norm_of_large_values_in_place(K, out_format):
    """The stream written over the residual: the second sum reads what was written."""
    g = gen(K)
    x, r = (torch.randn(7, K, generator=g) * 1e30).to(BF16), (torch.randn(7, K, generator=g) * 1e30).to(BF16)
    want = binding.svdq_add_rmsnorm(x.cuda(), torch.ones(K).cuda(), residual=r.cuda(), out_format=out_format)
    rc = r.cuda()
    got = binding.svdq_add_rmsnorm(x.cuda(), torch.ones(K).cuda(), residual=rc, residual_out=rc, out_format=out_format)
    assert all(torch.equal(a, b) for a, b in zip(want, got) if a is not None)
    y, _, _ = norm64(x, r, torch.ones(K), 1e-6, "same", K)
    if out_format == "same":
        check(got[0], y, (U[BF16] * 1.001 + (K / 64 + 16) * EPS32) * y.abs() + SMALL[BF16], "out")


# ------------------------------------------------------------------ product
@pytest.mark.parametrize("t,big", [(E4M3, 448), (E4M3, 256), (F16, 448), (BF16, 384)])
@pytest.mark.parametrize("M,N,K", [(3, 64, 1040), (20, 64, 1040), (40, 80, 4112), (64, 96, 1040), (70, 136, 1040),
                                   (70, 3072, 12288), (400, 600, 528), (500, 9201, 2064), (770, 9210, 2064),
                                   (4608, 4500, 528)])
def test_gemm_sums_beside_large_products(M, N, K, t, big):
    """Whole numbers from -2 to 2 beside pairs of large products that cancel.  Every partial sum is a
    whole number below 2^24, which fp32 holds in any order, and the results, below 2048, are exact
    in fp16: one lost bit of a small product shows."""
    g = gen(M + N + K)
    x = torch.randint(-2, 3, (M, K), generator=g).float()
    w = torch.randint(-2, 3, (N, K), generator=g).float()
    # four pairs of columns, each in an eight of its own
    cols = torch.randperm(K // 8, generator=g)[:8] * 8 + torch.randint(0, 8, (8,), generator=g)
    x[:, cols] = big
    w[:, cols[0::2]], w[:, cols[1::2]] = big, -big
    y = binding.svdq_gemm_act_residual(x.to(t).cuda(), w.to(t).cuda(), out_dtype=F16)
    want = x.cuda().to(F64) @ w.cuda().to(F64).T
    assert float(want.abs().max()) < 2048
    assert torch.equal(y.to(F64), want)


# ------------------------------------------------------------------ other streams
def block_calls():
    g = gen(21)
    x, r, w = (torch.randn(*s, generator=g).to(BF16).cuda() for s in ((70, 4096), (70, 4096), (96, 4096)))
    n, q, f = torch.ones(4096).cuda(), torch.randn(5, 4, 64, generator=g).to(F16).cuda(), torch.rand(32).cuda()
    pos = torch.arange(5, dtype=torch.int32).unsqueeze(-1).cuda()
    return [lambda s: binding.svdq_add_rmsnorm(x, n, residual=r, stream=s),
            lambda s: (binding.svdq_gemm_act_residual(x, w, stream=s),),            # K split: a workspace
            lambda s: binding.svdq_rope_axes(q, q, pos, f, (32,), stream=s)]


def test_calls_on_another_stream():
    """A stream's handle, and 0 for the default stream: the same bits, in memory that the current
    stream has not just freed."""
    assert binding.gemm_act_residual_workspace_bytes(70, 96, 4096, 1) > 0
    side = torch.cuda.Stream()
    for call in block_calls():
        want = call(None)
        torch.cuda.synchronize()
        for handle in (side.cuda_stream, 0):
            got = call(handle)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got))
        freed = {t.data_ptr() for t in call(None)}          # handed back to the current stream's pool
        got = call(side.cuda_stream)
        assert not freed & {t.data_ptr() for t in got}
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


# ------------------------------------------------------------------ rotary positions
def rope_both(q, pos, freq, axis_pairs, pairs="adjacent", inverse=False, **kw):
    """The operator on q as it is and on a copy one element off 16-byte alignment, which takes the
    element-wise kernel; both in the operator's layout, on the CPU."""
    buf = torch.zeros(q.numel() + 1, dtype=q.dtype, device="cuda")
    off = buf[1:].view(q.shape)
    off.copy_(q)
    return [binding.svdq_rope_axes(v, None, pos.cuda(), freq.cuda(), axis_pairs, pairs, inverse=inverse, **kw)[0].cpu()
            for v in (q.cuda(), off)]


def check_turned(q, pos, freq, axis_pairs, pairs):
    want, size = rope64(q, None, pos, freq, axis_pairs, pairs, 1e-6, False)
    # cosine and sine within 2^-21, two products and their difference, one rounding
    tol = U[q.dtype] * 1.001 * want.abs() + 2.0 ** -20 * size + SMALL[q.dtype]
    for y in rope_both(q, pos, freq, axis_pairs, pairs):
        check(y, want, tol, f"positions up to {float(pos.abs().max()):.3g}")


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("octave", list(range(18, 31)))
def test_rope_every_int_position(octave, pairs):
    """Positions of every size an int32 holds, both signs, with frequencies of one and below."""
    g = gen(octave)
    pos = torch.randint(1 << octave, (1 << (octave + 1)) - 1, (257, 1), generator=g, dtype=torch.int64)
    pos[0], pos[1] = 1 << octave, (1 << (octave + 1)) - 1
    pos[2::2] *= -1
    freq = torch.cat([torch.ones(1), torch.rand(31, generator=g)])
    check_turned(torch.randn(257, 2, 64, generator=g).to(F16), pos.to(torch.int32), freq, (32,), pairs)


@pytest.mark.parametrize("exponent", [20, 30, 36, 42, 47])
def test_rope_large_fp32_angles(exponent):
    g = gen(exponent)
    pos = (torch.rand(64, 1, generator=g) + 1) * 2.0 ** (exponent // 2) * (torch.randint(0, 2, (64, 1), generator=g) * 2 - 1)
    freq = (torch.rand(32, generator=g) + 1) * 2.0 ** ((exponent - 1) // 2)
    check_turned(torch.randn(64, 2, 64, generator=g).to(F16), pos, freq, (32,), "adjacent")


def test_rope_angles_past_the_limit():
    """Angles past 2^48, infinite ones too, are taken as 2^48 with their sign; NaN shows in its pair alone."""
    limit, q = 2.0 ** 48, torch.zeros(8, 1, 16, dtype=F16)
    q[..., 0::2] = 1                         # pairs (1, 0) become (cos, sin)
    values = [limit, limit * 1.5, 1e30, float("inf"), -limit, -1e30, float("-inf"), float("nan")]
    pos = torch.tensor([[v] for v in values])
    freq = torch.tensor([1.0] + [0.0] * 7)
    pos2 = torch.where(torch.isfinite(pos), pos, torch.zeros(()))      # 0 times an infinity is NaN too
    for y in rope_both(q, torch.cat([pos, pos2], -1), freq, (1, 7)):
        assert bool((y[:, 0, 2::2] == 1).all()) and bool((y[:, 0, 3::2] == 0).all())
        turned = y[:, 0, :2].double()
        want = torch.tensor([torch.cos(torch.tensor(limit, dtype=F64)), torch.sin(torch.tensor(limit, dtype=F64))])
        assert float((turned[0] - want).abs().max()) < 2.0 ** -11
        assert all(torch.equal(turned[i], turned[0]) for i in (1, 2, 3))
        for i in (4, 5, 6):
            assert float(turned[i, 0]) == float(turned[0, 0]) and float(turned[i, 1]) == -float(turned[0, 1])
        assert bool(torch.isnan(turned[7]).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("D,axis_pairs", [(128, (8, 24)), (64, (5,)), (72, (3, 4, 8)), (256, (60, 60)), (16, (1,))])
def test_rope_values_behind_the_pairs(D, axis_pairs, pairs, dtype):
    """Infinities, NaN and negative zeros behind the turned values stay where they are, bit for bit,
    and reach no neighbour; so do all other values there."""
    g, P = gen(D), sum(axis_pairs)
    q = torch.randn(130, 3, D, generator=g).to(dtype)
    pos = torch.randint(0, 5000, (130, len(axis_pairs)), generator=g, dtype=torch.int32)
    freq = torch.rand(P, generator=g)
    clean = rope_both(q, pos, freq, axis_pairs, pairs)
    odd = torch.tensor([float("inf"), float("nan"), -0.0, float("-inf"), 0.0, 1.0]).to(dtype)
    pick = torch.randint(0, len(odd), q[..., 2 * P:].shape, generator=g)
    q[..., 2 * P:] = odd[pick]
    for y, c in zip(rope_both(q, pos, freq, axis_pairs, pairs), clean):
        assert torch.equal(y[..., :2 * P], c[..., :2 * P])
        nan = torch.isnan(q[..., 2 * P:])
        assert torch.equal(torch.isnan(y[..., 2 * P:]), nan)
        assert torch.equal(y[..., 2 * P:][~nan].view(torch.int16), q[..., 2 * P:][~nan].view(torch.int16))


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("D", [1, 8, 64, 100, 128, 256])
def test_rope_norm_of_large_values(D, pairs):
    """Heads whose squares pass fp32's range beside ordinary ones."""
    if D == 1:
        D, P = 2, 1
    else:
        P = D // 2
    g = gen(D)
    scale = torch.tensor([1.0, 1e18, 2e19, 1e25, 3.0, 1e33, 1e37])[:, None, None]
    q = (torch.randn(7, 5, D, generator=g) * scale).to(BF16)
    w = 1 + 0.2 * torch.randn(D, generator=g)
    pos, freq = torch.arange(7, dtype=torch.int32)[:, None], torch.rand(P, generator=g)
    want, size = rope64(q, w, pos, freq, (P,), pairs, 1e-6, False)
    # the norm's sum and root, cosine and sine, one rounding
    tol = U[BF16] * 1.001 * want.abs() + (2.0 ** -20 + (D / 8 + 8) * EPS32) * size + SMALL[BF16]
    for y in rope_both(q, pos, freq, (P,), pairs, q_weight=w.cuda()):
        check(y, want, tol, f"heads of {D}")


@pytest.mark.parametrize("M", [16, 256])
def test_gemm_every_e4m3_code(M):
    """All 256 codes times one, as x and as w: fp16 holds each value, subnormal ones too, and NaN stays NaN."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(E4M3).view(16, 16).cuda()
    x = torch.zeros(M, 256, device="cuda").to(E4M3)
    x[:16, :16] = codes
    one = torch.eye(256, device="cuda").to(E4M3)
    value = codes.to(F16)
    got = binding.svdq_gemm_act_residual(x, one, out_dtype=F16)[:16, :16]
    nan = torch.isnan(value)                 # in x, NaN reaches its whole row
    assert int(nan.sum()) == 2 and bool(torch.isnan(got[nan.any(1)]).all())
    assert torch.equal(got[~nan.any(1)], value[~nan.any(1)])
    got = binding.svdq_gemm_act_residual(torch.eye(256, device="cuda")[:M].to(E4M3), x[:16].contiguous(), out_dtype=F16)[:16]
    assert torch.equal(got[:, ~nan.any(1)], value[~nan.any(1)].T) and bool(torch.isnan(got[:, nan.any(1)]).all())


@pytest.mark.parametrize("t,least,large", [(F16, -24, 10), (BF16, -133, 125), (E4M3, -9, 4)])
@pytest.mark.parametrize("M,N,K", [(3, 64, 1040), (70, 136, 1040), (520, 1100, 528), (4030, 3931, 160)])
def test_gemm_subnormal_operands(M, N, K, t, least, large):
    """Whole multiples of the type's smallest value: they count in full."""
    g = gen(M + K)
    x, w = torch.randint(-7, 8, (M, K), generator=g), torch.randint(-3, 4, (N, K), generator=g)
    xt, wt = (x.to(F64) * 2.0 ** least).to(t), (w.to(F64) * 2.0 ** large).to(t)
    assert torch.equal(xt.to(F64), x.to(F64) * 2.0 ** least)
    y = binding.svdq_gemm_act_residual(xt.cuda(), wt.cuda(), xs=torch.full((M,), 2.0 ** -(least + large)).cuda(), out_dtype=F16)
    assert torch.equal(y, (x.to(F64).cuda() @ w.to(F64).cuda().T).to(F16))
