"""The largest sizes svdq_tree_attention takes and those its workspace function knows are the same, without a GPU."""
import ctypes

import pytest

from bit_w4a4_quantized_amd import binding

NULL, SHAPE = -1, -2


def status(tokens, heads, kv, sequences):
    """Of a call without pointers: that of its sizes comes first."""
    c = binding.CacheStruct(type=0, pages=1, page_size=16, heads=kv, dim=64, page_stride=16 * kv * 64, token_stride=kv * 64,
                            head_stride=64)
    b = binding.BatchStruct(table_stride=4, table_width=4, sequences=sequences)
    return binding.lib().svdq_tree_attention(ctypes.addressof(c), ctypes.addressof(b), None, heads * 64, 64, heads, tokens, 0,
                                             1.0, None, 0, 0, None, heads * 64, 64, None, 0, None)


@pytest.mark.parametrize("tokens,heads,kv,sequences,fits", [
    ((1 << 20) - 1, 256, 1, 1, True), (1 << 20, 256, 1, 1, False), (1, 1 << 16, 1 << 16, 256, True),
    (1, 1 << 16, 1 << 16, 257, False), (16, 1 << 16, 1 << 16, 255, True), (16, 1 << 16, 1 << 16, 256, False),
    (1 << 24, 16, 1, 1, False), (1 << 15, 1 << 16, 1, 1, False), ((1 << 15) - 1, 1 << 16, 1 << 8, 1, False)])
def test_tiles(tokens, heads, kv, sequences, fits):
    assert status(tokens, heads, kv, sequences) == (NULL if fits else SHAPE)
    if not fits:
        assert binding.tree_attention_workspace_bytes(sequences, tokens, heads, kv, 64, 1 << 14, 1 << 16) == 0


def test_table():
    f = binding.tree_attention_workspace_bytes
    assert f(1, 1, 8, 8, 64, 1 << 14, 1 << 16) > 0 and f(1, 1, 8, 8, 64, (1 << 14) + 1, 1 << 16) == 0


@pytest.mark.parametrize("sequences,tokens,heads,kv,dim", [(1, 1, 32, 8, 128), (64, 64, 32, 8, 128), (3, 60, 8, 8, 256),
                                                           (2, 2000, 64, 64, 16), (1, 4096, 32, 8, 128), (5, 185, 24, 8, 80)])
def test_workspace_is_bounded(sequences, tokens, heads, kv, dim):
    """Parts are as many as fill the chip, not as many as a table has room for."""
    f = binding.tree_attention_workspace_bytes
    sizes = [f(sequences, tokens, heads, kv, dim, 1 << n, 64) for n in range(0, 25)]
    assert sizes == sorted(sizes) and sizes[-1] <= 256 << 20
