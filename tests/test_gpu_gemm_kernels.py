"""Every kernel of svdq_gemm_act_residual in every type, at ragged sizes that are checked to reach it,
against the product in 64 bits (tolerances of test_gpu_block.py)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_w4a4_quantized_amd import binding  # noqa: E402
from gemm_kernels import CASES, TYPE_CODES  # noqa: E402
from test_gpu_block import BF16, E4M3, F16, _gpu, gemm_case  # noqa: E402, F401

TYPES = {"int8": torch.int8, "e4m3": E4M3, "f16": F16, "bf16": BF16}


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("kernel,split,tail,size", CASES)
def test_gemm_kernel(kernel, split, tail, size, t):
    name, splits, cut = binding.gemm_act_residual_kernel(*size, TYPE_CODES[t])
    assert (name, splits > 1, cut) == (kernel, split, tail)
    gemm_case(*size, TYPES[t], BF16, "silu", ypad=3)
    if kernel != "few rows":
        return
    gemm_case(*size, TYPES[t], F16, "gelu", inplace=True)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("kernel,split,tail,size", [c for c in CASES if c[0] != "few rows"][::2])
def test_gemm_kernel_residual_in_place(kernel, split, tail, size, t):
    """y is the residual: each kernel reads it before it writes there."""
    gemm_case(*size, TYPES[t], F16, "gelu", bias=False, inplace=True)


@pytest.mark.parametrize("t", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("kernel,split,tail,size", [c for c in CASES if c[0] != "few rows"])
def test_gemm_kernel_not_finite(kernel, split, tail, size, t):
    """NaN behind x's rows reaches nothing; in x, w or the residual its own row, column or element."""
    M, N, K = size
    dt, g = TYPES[t], torch.Generator(device="cuda").manual_seed(M + N)
    xb, w = torch.randn(M, K + 16, generator=g, device="cuda").to(dt), torch.randn(N, K, generator=g, device="cuda").to(dt)
    r = torch.randn(M, N, generator=g, device="cuda").to(F16)
    run = lambda: binding.svdq_gemm_act_residual(xb[:, :K], w, residual=r, out_dtype=F16)  # noqa: E731
    clean = run()
    assert bool(torch.isfinite(clean).all())
    xb[:, K:] = float("nan")
    xb[2, K - 1] = float("nan")
    w[N - 1, 0] = float("nan")
    r[0, 1] = float("nan")
    got, want = run(), torch.zeros(M, N, dtype=torch.bool, device="cuda")
    want[2], want[:, N - 1], want[0, 1] = True, True, True
    assert torch.equal(torch.isnan(got), want)
    assert torch.equal(got[~want], clean[~want])
