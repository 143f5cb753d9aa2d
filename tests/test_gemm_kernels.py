"""Which kernel svdq_gemm_act_residual takes, without a GPU: the sizes of the GPU tests reach the kernels
they are meant for (256 CUs, the number taken where there is no GPU)."""
import pytest

torch = pytest.importorskip("torch")

from bit_w4a4_quantized_amd import binding  # noqa: E402
from gemm_kernels import CASES, TYPE_CODES  # noqa: E402


@pytest.mark.parametrize("t", TYPE_CODES)
@pytest.mark.parametrize("kernel,split,tail,size", CASES)
def test_sizes_reach_their_kernel(kernel, split, tail, size, t):
    name, splits, cut = binding.gemm_act_residual_kernel(*size, TYPE_CODES[t])
    assert (name, splits > 1, cut) == (kernel, split, tail)
    whole_tiles = -(-size[0] // 256) * -(-size[1] // 256)
    if kernel == "256x256":
        assert (tail == 0) == (whole_tiles % 256 == 0)


def test_every_kernel_has_a_size():
    assert {(k, s, c) for k, s, c, _ in CASES} == {
        ("few rows", False, 0), ("64x64", False, 0), ("64x64", True, 0), ("64x128", False, 0), ("64x128", True, 0),
        ("128x192", False, 0), ("128x256", False, 0), ("256x256", False, 0), ("256x256", False, 1), ("256x256", False, 2),
        ("256x256", False, 4)}


def test_less_workspace_splits_less():
    for t, code in TYPE_CODES.items():
        M, N, K = 68, 56, 4016
        need = binding.gemm_act_residual_workspace_bytes(M, N, K, code)
        assert need > 0 and binding.gemm_act_residual_kernel(M, N, K, code, 0)[1] == 1
        assert 1 < binding.gemm_act_residual_kernel(M, N, K, code, need - 1)[1] < binding.gemm_act_residual_kernel(
            M, N, K, code)[1]


def test_query_refusals():
    assert binding.gemm_act_residual_kernel(4, 32, 64, 3)[0] == "few rows"
    for bad in ((-1, 32, 64, 3), (4, -1, 64, 3), (4, 32, 0, 3), (4, 32, 40, 3), (4, 32, 64, 2), (4, 32, 64, 5), (4, 32, 60, 0),
                (0, 32, 64, 3), (4, 0, 64, 3)):
        assert binding.gemm_act_residual_kernel(*bad, 0) is None
    assert binding.lib().svdq_gemm_act_residual_kernel(4, 32, 64, 3, 0, None, None) == b"few rows"
