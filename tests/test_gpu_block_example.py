"""examples/transformer_block.py: the block operators and the W4A4 layers together, two blocks deep,
against the same blocks from the unquantized weights.

Bounds: a symmetric b-bit code of a group of normal values is off by about a / qmax / sqrt(12) with a
the group's maximum, 2.5 to 3.5 standard deviations: 0.14 of a value's size for 4 bits (a / sigma =
2.5 for 64 values, qmax 7) on each of a W4A4 layer's operands, so 0.15 to 0.2 per layer on what its
low-rank branch leaves, and about 0.3 through the pair and its GELU.  The stream adds these branches
to values of their size or larger: half that, and 8 bits add a hundredth."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("side,text", [(8, 13), (1, 0)])
def test_transformer_block(side, text):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import transformer_block
    stream, mlp = transformer_block.main(512, 4, 2048, (16, 24, 24), text, side, 2, check=True)
    print(f"stream off by {stream:.3g}, MLP output by {mlp:.3g}")
    assert stream < 0.15 and mlp < 0.3
