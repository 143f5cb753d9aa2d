"""examples/transformer_block.py over paged caches: prompts, a drafted tree, its accepted path and one more token run
through two blocks."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("prompts,axis_pairs", [((70, 1, 130), (64,)), ((5,), (16, 24, 24))])
def test_cached_block(prompts, axis_pairs):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import transformer_block
    out = transformer_block.cached(512, 4, 2048, axis_pairs, prompts)
    assert out.shape == (len(prompts), 512) and bool(torch.isfinite(out).all())
