"""A required tensor that is missing is refused like a wrong one, with ValueError and its name."""
import pytest

torch = pytest.importorskip("torch")

from bit_w4a4_quantized_amd import binding  # noqa: E402
from test_block_checks import gemm_args, norm_args, rec, rope_args  # noqa: E402, F401

CALLS = {"svdq_add_rmsnorm": (norm_args, ("x", "weight")), "svdq_gemm_act_residual": (gemm_args, ("x", "w")),
         "svdq_rope_axes": (rope_args, ("q", "positions", "inv_freq"))}


@pytest.mark.parametrize("fn,missing", [(f, m) for f, (_, names) in CALLS.items() for m in names])
def test_missing_tensors(fn, missing, rec):  # noqa: F811
    with pytest.raises(ValueError, match=missing):
        getattr(binding, fn)(**CALLS[fn][0](**{missing: None}))
    assert not rec.calls
