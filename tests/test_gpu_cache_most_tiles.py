"""svdq_tree_attention at the most tiles it takes, 2^24: a batch padded to 256 sequences of 2^16 heads."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_w4a4_quantized_amd import binding  # noqa: E402
from test_gpu_cache import F16, _gpu, gen, randn  # noqa: E402, F401


@pytest.mark.parametrize("sequences", [255, 256])
def test_most_tiles(sequences):
    heads, dim, mine = 1 << 16, 8, 200
    g = gen(151)
    k, v = (randn(g, 3, 1, heads, dim).to(F16).cuda() for _ in range(2))
    q = randn(g, 1, heads, dim).to(F16).cuda()
    table = torch.full((sequences, 1), -1, dtype=torch.int32, device="cuda")
    table[mine] = 1
    starts = (torch.arange(sequences + 1, device="cuda") > mine).int()
    batch = binding.PagedBatch(table, starts, torch.zeros(sequences, dtype=torch.int32, device="cuda"))
    out = binding.svdq_tree_attention(binding.PagedCache(k, v), batch, q)
    torch.cuda.synchronize()
    assert torch.equal(out[0], v[1, 0])      # one token that sees itself
