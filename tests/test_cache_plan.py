"""The workspace svdq_tree_attention asks for, over dense sweeps of its sizes, without a GPU: the sums of at most a few
rounds of workgroups, whatever the sequences' number is next to a round's."""
import pytest

from bit_w4a4_quantized_amd import binding

BOUND = 256 << 20


@pytest.mark.parametrize("heads,kv,dim", [(32, 8, 128), (64, 8, 128), (8, 4, 256), (24, 24, 80), (16, 16, 64), (8, 1, 256), (1, 1, 64)])
@pytest.mark.parametrize("table", [512, 2048, 32768, 131072, 1 << 20])
def test_bytes_bounded(heads, kv, dim, table):
    f = binding.lib().svdq_tree_attention_workspace_bytes
    worst = (0,)
    for each in (1, 2, 5, 9, 16, 17, 32, 33, 61, 64, 128, 129, 500, 4096):
        for sequences in [*range(1, 140), *range(140, 1100, 7), 255, 256, 257, 511, 512, 513, 1023, 1024, 1025]:
            n = f(sequences, each * sequences, heads, kv, dim, table // 64, 64)
            worst = max(worst, (n, sequences, each))
    assert worst[0] <= BOUND, f"{worst[0]} bytes for {worst[1]} sequences of {worst[2]}"


@pytest.mark.parametrize("heads,kv,dim,each", [(32, 8, 128, 9), (32, 8, 128, 16), (64, 8, 128, 9), (8, 4, 256, 64)])
def test_no_cliff(heads, kv, dim, each):
    """One sequence more does not multiply the workgroups: parts of the last, partial round of tiles alone."""
    f = binding.lib().svdq_tree_attention_workspace_bytes
    one = 128 * (dim + 2) * 4                # a part's sums
    for sequences in range(1, 1100):
        assert f(sequences, each * sequences, heads, kv, dim, 512, 64) <= 3 * 512 * one
