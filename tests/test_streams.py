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


# ------------------------------------------------------------------ the W4A4 layer and its parts
M, K, N, R = 8, 128, 64, 16
FMT = "int4_e2m3"


def codes(rows, fmt=FMT):
    return T(binding.code_shape(rows, K, fmt), torch.uint8), T(binding.scale_shape(rows, K, fmt), binding.scale_dtype(fmt))


def half(*shape):
    return T(shape, F16)


def layer():
    return half(R, K), *codes(N), half(R, N), half(N)


LAYER = {
    "quantize_down": (4, lambda s: binding.svdq_quantize_down(half(M, K), half(R, K), FMT, stream=s)),
    "quantize_down_smooth": (4, lambda s: binding.svdq_quantize_down_smooth(half(M, K), T((K,), F32), half(R, K), FMT, stream=s)),
    "gemm_up": (1, lambda s: binding.svdq_gemm_w4a4_up(*codes(M), half(M, R), *codes(N), half(R, N), None, K, FMT, stream=s)),
    "gemm_up_gelu": (1, lambda s: binding.svdq_gemm_w4a4_up_gelu_smooth(*codes(M), half(M, R), *codes(N), half(R, N), None,
                                                                        T((N,), F32), K, FMT, stream=s)),
    "linear": (2, lambda s: binding.svdq_linear(half(M, K), *layer(), FMT, stream=s)),
    "linear_unfused": (2, lambda s: binding.svdq_linear_unfused(half(M, K), *layer(), FMT, stream=s)),
    "linear_folded": (2, lambda s: binding.svdq_linear_folded(half(M, K), None, *layer(), None, FMT, stream=s)),
    "quantize_weight": (2, lambda s: binding.svdq_quantize_weight(T((N, K), F32), FMT, stream=s)),
    "pack_weight": (2, lambda s: binding.svdq_pack_weight(T((N, K), I8), half(N, K // 64), FMT, stream=s)),
    "w4a16": (1, lambda s: binding.svdq_gemm_w4a16(half(M, K), *codes(N, "int4"), None, stream=s)),
    "gelu": (1, lambda s: binding.svdq_gelu_tanh_smooth(half(M, N), T((N,), F32), stream=s)),
    "relayout": (2, lambda s: binding.svdq_relayout(*codes(N), K, FMT, True, stream=s)),
}


@pytest.fixture
def layer_made(made, monkeypatch):
    for f in ("linear_workspace_bytes", "linear_unfused_workspace_bytes", "quantize_down_workspace_bytes"):
        monkeypatch.setattr(binding, f, lambda *a: 4096)
    return made


@pytest.mark.parametrize("op", LAYER)
def test_layer_allocates_on_the_launch_stream(op, layer_made, rec):  # noqa: F811
    count, call = LAYER[op]
    out = call(SIDE)
    assert len(layer_made) == count and all(t.under == SIDE for t in layer_made)
    assert rec.calls[-1][1][-1] == SIDE
    assert all(t.recorded == ["current"] for t in (out if isinstance(out, tuple) else (out,)))


def test_prepared_layer_keeps_a_workspace_for_each_stream(layer_made, rec):  # noqa: F811
    """Calls on two streams may run at once: they share no workspace, and each is of its stream's pool."""
    l1t, wq, ws, l2, bias = layer()
    net = binding.SvdqLinear(wq, ws, l1t, l2, bias, K, FMT)
    net._raw_stream = lambda dev: 7
    net(half(M, K))
    assert [t.under for t in layer_made] == ["current"] * 2
    net(half(M, K), stream=SIDE)
    assert [t.under for t in layer_made[2:]] == [SIDE] * 2
    net(half(M, K), y=half(M, N), stream=SIDE)
    net(half(M, K), y=half(M, N))
    assert len(layer_made) == 4              # both kept
    net(half(2 * M, K), y=half(2 * M, N), stream=SIDE)
    assert [t.under for t in layer_made[4:]] == [SIDE]
