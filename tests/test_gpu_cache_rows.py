"""svdq_tree_attention over batches whose starts fall: rows of no sequence and what lies around q and out stay as they
were.  Heads outermost, so that a row of another head would lie far from its token."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_w4a4_quantized_amd import binding  # noqa: E402
from test_gpu_cache import E4M3, F16, I8, Pages, _gpu, gen, randn  # noqa: E402, F401


@pytest.mark.parametrize("cache", [F16, I8, E4M3])
@pytest.mark.parametrize("heads", [2, 8])
@pytest.mark.parametrize("starts", [(40, 0, 7, 20), (45, 45, 0, 3), (30, 10, 10, 12), (44, 1, 2, 2), (20, 40, 3, 5)])
def test_falling_starts(starts, heads, cache):
    g = gen(71)
    p = Pages(g, [15, 15, 15], [30, 20, 9], 1, 64, cache, 8)
    batch = binding.PagedBatch(p.batch.page_table, torch.tensor(starts, dtype=torch.int32).cuda(), p.batch.context)
    q = randn(g, heads + 2, 45, 64).to(F16).cuda()[1:-1].transpose(0, 1)
    tree = torch.ones(45, 45, dtype=torch.bool, device="cuda")
    of_one = torch.zeros(45, dtype=torch.bool)
    for s0, s1 in zip(starts, starts[1:]):
        of_one[s0:max(s0, s1)] = True
    for t in (None, tree):
        buf = torch.full((heads + 2, 45, 64), 4.0, dtype=F16, device="cuda")
        out = buf[1:-1].transpose(0, 1)
        binding.svdq_tree_attention(p.cache, batch, q, tree=t, out=out)
        torch.cuda.synchronize()
        assert bool((buf[0] == 4).all()) and bool((buf[-1] == 4).all())
        assert bool((out.cpu()[~of_one] == 4).all())         # what the rows of such sequences hold is open
