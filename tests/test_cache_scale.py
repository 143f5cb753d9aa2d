"""The scales of logits that svdq_tree_attention takes, without a GPU: those whose product with log2(e) is a
normal fp32 number."""
import ctypes

import pytest

from bit_w4a4_quantized_amd import binding

NULL, SHAPE = -1, -2


@pytest.mark.parametrize("scale,status", [(2.0 ** -127, SHAPE), (2.0 ** -126, NULL), (1e-30, NULL), (1.0, NULL), (1e30, NULL),
                                          (2.0 ** 126, NULL), (2.0 ** 127, SHAPE), (3.0e38, SHAPE), (1e-45, SHAPE), (-1.0, SHAPE)])
def test_scale(scale, status):
    c = binding.CacheStruct(type=0, pages=1, page_size=16, heads=1, dim=64, page_stride=1024, token_stride=64, head_stride=64)
    b = binding.BatchStruct(table_stride=4, table_width=4, sequences=1)
    assert binding.lib().svdq_tree_attention(ctypes.addressof(c), ctypes.addressof(b), None, 64, 64, 1, 1, 0, scale, None, 0, 0,
                                             None, 64, 64, None, 0, None) == status
