"""Where the binding allocates when a call names another stream, on the CPU with stand-ins: memory
that a call writes on a stream has to come from that stream's pool.  A block of the current stream's
pool may still be in use there when the allocator hands it out, and nothing orders the other stream
behind that use."""
import contextlib
import functools

import pytest

torch = pytest.importorskip("torch")

from bit_w4a4_quantized_amd import binding  # noqa: E402
from test_block_checks import Dev, rec  # noqa: E402, F401

F16, BF16, F32, I8 = torch.float16, torch.bfloat16, torch.float32, torch.int8
SIDE = 1234


meta_empty = torch.empty


class T(Dev):
    """A stand-in whose shape is a torch.Size, made without torch.empty."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.is_cuda, self.device = torch.Size(shape), dtype, True, torch.device("cuda:0")
        self._t = meta_empty(shape, dtype=dtype, device="meta")

    def numel(self):
        return self._t.numel()

    def element_size(self):
        return self._t.element_size()

    def new_empty(self, shape):
        return torch.empty(shape, dtype=self.dtype, device=self.device)

    def record_stream(self, s):
        self.recorded.append(s)


@pytest.fixture
def made(monkeypatch, rec):  # noqa: F811
    """The tensors allocated by a call, with the stream each was made under; rec.calls has the launches."""
    out, now = [], ["current"]

    def empty(shape, dtype=None, device=None):
        t = T(shape if isinstance(shape, (tuple, list)) else (shape,), dtype)
        t.under, t.recorded = now[-1], []
        out.append(t)
        return t

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: empty(t.shape, t.dtype))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device=None: s)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(binding, "gemm_act_residual_workspace_bytes", functools.lru_cache(lambda *a: 4096))
    return out


BLOCK = {
    "norm": lambda s: binding.svdq_add_rmsnorm(T((4, 64), BF16), T((64,), F32), residual=T((4, 64), F32), stream=s),
    "gemm": lambda s: binding.svdq_gemm_act_residual(T((4, 64), I8), T((32, 64), I8), stream=s),
    "rope": lambda s: binding.svdq_rope_axes(T((5, 4, 64), F16), T((5, 2, 64), F16), T((5, 1), torch.int32),
                                             T((32,), F32), (32,), heads_first=True, stream=s),
}
MADE = {"norm": 3, "gemm": 2, "rope": 2}


@pytest.mark.parametrize("op", BLOCK)
def test_block_operators_allocate_on_the_launch_stream(op, made, rec):  # noqa: F811
    out = BLOCK[op](SIDE)
    assert len(made) == MADE[op] and all(t.under == SIDE for t in made)
    assert rec.calls[-1][1][-1] == SIDE
    # what the caller gets may be used and freed on its own stream
    for t in out if isinstance(out, tuple) else (out,):
        assert t.recorded == ["current"]


@pytest.mark.parametrize("op", BLOCK)
def test_block_operators_on_the_current_stream(op, made, rec):  # noqa: F811
    BLOCK[op](None)
    assert len(made) == MADE[op] and all(t.under == "current" and not t.recorded for t in made)
    assert rec.calls[-1][1][-1] == 7
