"""svdq_tree_attention with page tables far wider than the contexts, as a server's are: the keys' parts are cut for the
table's width, and those past a context's end are neither computed nor joined."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_w4a4_quantized_amd import binding  # noqa: E402
from strict import check  # noqa: E402
from test_gpu_cache import BF16, E4M3, F16, I8, QMAX, U, Pages, _gpu, attend, attention64, gen, randn, random_tree  # noqa: E402, F401


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (F16, I8), (BF16, E4M3)])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("counts,contexts,heads,kv,dim", [([1], [999], 8, 2, 128), ([1, 0, 2], [70, 5, 0], 4, 2, 64), ([12, 3], [300, 1], 4, 2, 128),
                                                          ([100], [500], 2, 1, 128), ([60, 61, 1], [200, 0, 64], 2, 1, 256)])
def test_wide_table(counts, contexts, heads, kv, dim, tree, dtype, cache):
    g = gen(141 + sum(counts))
    p = Pages(g, counts, contexts, kv, dim, cache, 16)
    q = (2 * randn(g, p.tokens, heads, dim)).to(dtype)
    t = random_tree(g, counts) if tree else None
    want, tol = attention64(p, q, t, dim ** -0.5, U[F16] if cache in QMAX else U[dtype])
    p.table = torch.cat([p.table, torch.full((len(counts), 8192 - p.width), -1, dtype=torch.int32)], 1)
    p.width = 8192
    p.upload()
    need = binding.tree_attention_workspace_bytes(len(counts), p.tokens, heads, kv, dim, 8192, 16)
    workspace = torch.full((need,), 123, dtype=torch.uint8, device="cuda")
    check(attend(p, q, t, workspace=workspace), want, tol, "a wide table")
    # parts for 131072 keys are more than the contexts have pieces of 64
    assert need > 0 and bool((workspace[:need // 2] == 123).any()) and float((workspace == 123).float().mean()) > 0.5
    workspace.fill_(255)                     # NaN where no part has been: not joined
    check(attend(p, q, t, workspace=workspace), want, tol, "a wide table, NaN in the workspace")
