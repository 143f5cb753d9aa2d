"""The block operators at the edges of their definitions: sums of products of very different sizes,
and whatever else an ordinary input does not show.  Exact where the definition is."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_w4a4_quantized_amd import binding  # noqa: E402

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
