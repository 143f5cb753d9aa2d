"""Refusals of the block operators (svdq_add_rmsnorm, svdq_gemm_act_residual, svdq_rope_axes), on
the CPU: the C ABI's status codes, returned before any HIP call, and the binding's argument
checks, raised before the library is called; and the offline weights and frequencies."""
import ctypes
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

from bit_w4a4_quantized_amd import binding, prepare  # noqa: E402
from bit_w4a4_quantized_amd.binding import RopeOperand  # noqa: E402

OK, NULL, SHAPE, ALIGN, FORMAT = 0, -1, -2, -3, -4
P, ODD, EIGHT = 4096, 4097, 4104          # fake pointers, never dereferenced on these paths
T16, TB, T32, I8, E4 = 0, 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


def norm(x=P, xst=64, xt=T16, r=P, rst=64, rt=T16, w=P, wt=T32, eps=1e-6, M=4, K=64, ot=I8, out=P, s=P, ro=P, rost=64):
    return binding.lib().svdq_add_rmsnorm(x, xst, xt, r, rst, rt, w, wt, eps, M, K, ot, out, s, ro, rost, None)


@pytest.mark.parametrize("bad,status", [
    (dict(xt=T32), FORMAT), (dict(xt=9), FORMAT), (dict(xt=-5), FORMAT), (dict(rt=TB), FORMAT), (dict(wt=TB), FORMAT),
    (dict(ot=TB), FORMAT), (dict(ot=T32), FORMAT), (dict(ot=7), FORMAT),
    (dict(M=-1), SHAPE), (dict(M=(1 << 24) + 1), SHAPE), (dict(K=0), SHAPE), (dict(K=-64), SHAPE),
    (dict(eps=0.0), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE), (dict(eps=INF), SHAPE),
    (dict(xst=63), SHAPE), (dict(rst=63), SHAPE), (dict(rost=63), SHAPE), (dict(xst=1 << 41), SHAPE),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL), (dict(s=None), NULL), (dict(ro=None), NULL),
    (dict(x=ODD), ALIGN), (dict(w=4098), ALIGN), (dict(s=4098), ALIGN), (dict(r=ODD), ALIGN), (dict(ro=ODD), ALIGN),
    (dict(rt=T32, r=4098), ALIGN), (dict(ot=T16, out=ODD), ALIGN),
    (dict(M=0, x=None, r=None, w=None, out=None, s=None, ro=None), OK), (dict(M=0, K=0), SHAPE),
])
def test_norm_statuses(bad, status):
    assert norm(**bad) == status


def gemm(x=P, xst=64, xs=P, w=P, ws=P, b=P, r=P, rst=32, M=4, N=32, K=64, t=I8, act=0, ot=T16, y=P, yst=32, wsp=P, wb=0):
    return binding.lib().svdq_gemm_act_residual(x, xst, xs, w, ws, b, r, rst, M, N, K, t, act, ot, y, yst, wsp, wb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(t=T32), FORMAT), (dict(t=5), FORMAT), (dict(ot=T32), FORMAT), (dict(ot=I8), FORMAT), (dict(act=3), FORMAT),
    (dict(act=-1), FORMAT), (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(N=(1 << 24) + 1), SHAPE), (dict(K=0), SHAPE),
    (dict(K=40), SHAPE), (dict(t=T16, K=60), SHAPE), (dict(xst=63), SHAPE), (dict(xst=72), SHAPE),
    (dict(K=(1 << 17) + 16, xst=1 << 20), SHAPE), (dict(t=E4, K=(1 << 22) + 16, xst=1 << 23), SHAPE),
    (dict(xst=(1 << 22) + 16), SHAPE), (dict(yst=31), SHAPE), (dict(rst=31), SHAPE),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL),
    (dict(x=EIGHT), ALIGN), (dict(w=EIGHT), ALIGN), (dict(y=ODD), ALIGN), (dict(xs=4098), ALIGN), (dict(ws=4098), ALIGN),
    (dict(b=ODD), ALIGN), (dict(r=ODD), ALIGN), (dict(wsp=EIGHT), ALIGN),
    (dict(M=0, x=None, w=None, y=None), OK), (dict(N=0, w=None, y=None, yst=0, rst=0), OK),
])
def test_gemm_statuses(bad, status):
    assert gemm(**bad) == status


def rope(count=2, B=1, T=4, D=64, t=T16, pos=P, pf=0, pb=0, f=P, axes=(8, 24), halves=0, eps=1e-6, inv=0, ops=P,
         n_axes=None, **op):
    one = dict(inp=P, out=P, weight=None, heads=2, in_batch=512, in_token=128, in_head=64, out_batch=512, out_token=128,
               out_head=64)
    arr = (RopeOperand * 2)(RopeOperand(**one), RopeOperand(**dict(one, **op)))
    ax = (ctypes.c_int * 8)(*axes) if axes is not None else None
    n = (len(axes) if axes is not None else 1) if n_axes is None else n_axes
    return binding.lib().svdq_rope_axes(ctypes.addressof(arr) if ops else None, count, B, T, D, t, pos, pf, pb, f, n, ax,
                                        halves, eps, inv, None)


@pytest.mark.parametrize("bad,status", [
    (dict(t=T32), FORMAT), (dict(t=I8), FORMAT), (dict(ops=None), NULL), (dict(axes=None), NULL),
    (dict(count=0), SHAPE), (dict(count=3), SHAPE), (dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(D=0), SHAPE),
    (dict(D=1025), SHAPE), (dict(n_axes=0), SHAPE), (dict(n_axes=5), SHAPE), (dict(axes=(8, 25)), SHAPE),
    (dict(axes=(-1, 8)), SHAPE), (dict(axes=(0, 0)), SHAPE), (dict(axes=(2000000000, 2000000000)), SHAPE),
    (dict(pb=-1), SHAPE), (dict(heads=0), SHAPE), (dict(in_batch=-1), SHAPE), (dict(out_head=1 << 41), SHAPE),
    (dict(weight=P, eps=0.0), SHAPE), (dict(weight=P, eps=NAN), SHAPE), (dict(weight=P, inv=1), FORMAT),
    (dict(B=1 << 16, T=1 << 16), SHAPE), (dict(B=1 << 10, T=1 << 18, heads=1 << 12), SHAPE),
    (dict(pos=None), NULL), (dict(f=None), NULL), (dict(inp=None), NULL), (dict(out=None), NULL),
    (dict(pos=4098), ALIGN), (dict(f=4098), ALIGN), (dict(inp=ODD), ALIGN), (dict(out=ODD), ALIGN),
    (dict(weight=4098), ALIGN), (dict(B=0, pos=None, f=None, inp=None, out=None), OK), (dict(T=0), OK),
])
def test_rope_statuses(bad, status):
    assert rope(**bad) == status


def test_sizes_past_one_launch():
    """A launch holds fewer than 2^32 threads; sizes that need more are refused, not cut."""
    assert norm(M=1 << 24, K=4096, rt=T32, xst=4096, rst=4096, rost=4096) == SHAPE
    assert norm(M=1 << 23, K=40000, r=None, xst=40000) == SHAPE
    assert rope(T=1 << 24, D=6, axes=(3,), heads=14) == SHAPE
    assert rope(B=1 << 6, T=1 << 24, D=1024, axes=(512,), heads=1) == SHAPE


# ------------------------------------------------------------------ the binding
class Dev:
    """A stand-in for a device tensor: shape, dtype, strides and a fake data pointer."""

    def __init__(self, shape, dtype, stride=None, cuda=True, device="cuda:0"):
        self.shape, self.dtype, self.is_cuda, self.device = tuple(shape), dtype, cuda, torch.device(device)
        self._t = torch.empty(shape, dtype=dtype, device="meta")
        if stride is not None:
            self._t = torch.empty_strided(shape, stride, dtype=dtype, device="meta")

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self._t.stride()

    def is_contiguous(self):
        return self._t.is_contiguous()

    def data_ptr(self):
        return P

    def get_device(self):
        return self.device.index


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            if not name.endswith("_bytes"):          # size queries: nothing needed
                self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(binding, "lib", lambda: r)
    monkeypatch.setattr(binding._d(), "raw_stream", lambda dev: 7)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    binding.gemm_act_residual_workspace_bytes.cache_clear()
    yield r
    binding.gemm_act_residual_workspace_bytes.cache_clear()


F16, BF16, F32, I8T = torch.float16, torch.bfloat16, torch.float32, torch.int8


def norm_args(**kw):
    a = dict(x=Dev((4, 64), BF16, (80, 1)), weight=Dev((64,), F32), residual=Dev((4, 64), F32),
             out=Dev((4, 64), I8T), scales=Dev((4,), F32), residual_out=Dev((4, 64), F32, (72, 1)))
    return {**a, **kw}


def test_norm_binding(rec):
    binding.svdq_add_rmsnorm(**norm_args())
    (name, args), = rec.calls
    assert name == "svdq_add_rmsnorm" and args == (P, 80, 1, P, 64, 2, P, 2, 1e-6, 4, 64, 3, P, P, P, 72, 7)
    for bad in (dict(x=None), dict(x=Dev((4, 64), F32)), dict(x=Dev((4, 64), BF16, cuda=False)), dict(x=Dev((64,), BF16)),
                dict(x=Dev((4, 64), BF16, (1, 4))), dict(x=Dev((4, 64), BF16, (32, 1))), dict(weight=Dev((63,), F32)),
                dict(weight=Dev((64,), F16)), dict(weight=Dev((64,), F32, (2,))), dict(residual=Dev((4, 65), F32)),
                dict(residual=Dev((4, 64), F16)), dict(residual=None), dict(residual_out=Dev((4, 64), BF16)),
                dict(residual_out=Dev((4, 64), F32, (0, 1))), dict(out=Dev((4, 64), F16)), dict(out=Dev((4, 64), I8T, (65, 1))),
                dict(scales=Dev((5,), F32)), dict(scales=Dev((4,), F16)), dict(out_format="fp4"), dict(out_format="same"),
                dict(scales=Dev((4,), F32, device="cuda:1"))):
        with pytest.raises(ValueError):
            binding.svdq_add_rmsnorm(**norm_args(**bad))
    assert len(rec.calls) == 1


def gemm_args(**kw):
    a = dict(x=Dev((4, 64), I8T, (80, 1)), w=Dev((32, 64), I8T), xs=Dev((4,), F32), ws=Dev((32,), F32),
             bias=Dev((32,), F16), activation="gelu", residual=Dev((4, 32), F16, (40, 1)), y=Dev((4, 32), F16))
    return {**a, **kw}


def test_gemm_binding(rec):
    binding.svdq_gemm_act_residual(**gemm_args())
    (name, args), = rec.calls
    assert name == "svdq_gemm_act_residual" and args == (P, 80, P, P, P, P, P, 40, 4, 32, 64, 3, 1, 0, P, 32, None, 0, 7)
    for bad in (dict(x=None), dict(x=Dev((4, 64), F32)), dict(x=Dev((4, 64), I8T, (1, 4))), dict(w=None),
                dict(w=Dev((32, 48), I8T)), dict(w=Dev((32, 64), F16)), dict(w=Dev((32, 64), I8T, (80, 1))),
                dict(xs=Dev((5,), F32)), dict(xs=Dev((4,), F16)), dict(ws=Dev((31,), F32)), dict(ws=Dev((32, 1), F32)),
                dict(bias=Dev((32,), F32)), dict(bias=Dev((33,), F16)), dict(activation="relu"), dict(out_dtype=F32),
                dict(out_dtype=BF16), dict(residual=Dev((4, 32), BF16)), dict(residual=Dev((4, 33), F16)),
                dict(y=Dev((4, 32), F32)), dict(y=Dev((3, 32), F16)), dict(y=Dev((4, 32), F16, (16, 1))),
                dict(w=Dev((32, 64), I8T, device="cuda:1"))):
        with pytest.raises(ValueError):
            binding.svdq_gemm_act_residual(**gemm_args(**bad))
    assert len(rec.calls) == 1


def rope_args(**kw):
    a = dict(q=Dev((2, 5, 4, 64), F16, (5 * 512, 512, 64, 1)), k=Dev((2, 5, 2, 64), F16), positions=Dev((5, 2), torch.int32),
             inv_freq=Dev((32,), F32), axis_pairs=(8, 24), q_weight=Dev((64,), F32), k_weight=Dev((64,), F32),
             q_out=Dev((2, 5, 4, 64), F16), k_out=Dev((2, 5, 2, 64), F16))
    return {**a, **kw}


def test_rope_binding(rec):
    binding.svdq_rope_axes(**rope_args())
    binding.svdq_rope_axes(**rope_args(positions=Dev((2, 5, 2), F32), heads_first=True, q_out=Dev((2, 4, 5, 64), F16),
                                       k_out=Dev((2, 2, 5, 64), F16)))
    assert [c[0] for c in rec.calls] == ["svdq_rope_axes"] * 2
    assert rec.calls[0][1][1:9] == (2, 2, 5, 64, 0, P, 0, 0) and rec.calls[1][1][6:9] == (P, 1, 10)
    for bad in (dict(q=None), dict(q=Dev((2, 5, 4, 64), F32)), dict(q=Dev((5, 4, 64), F16)), dict(q=Dev((5, 64), F16)),
                dict(q=Dev((2, 5, 4, 64), F16, (1280, 256, 1, 4))), dict(k=Dev((2, 6, 2, 64), F16)),
                dict(k=Dev((2, 5, 2, 64), BF16)), dict(k=None), dict(positions=Dev((4, 2), torch.int32)),
                dict(positions=Dev((5, 3), torch.int32)), dict(positions=Dev((5, 2), torch.int64)),
                dict(positions=Dev((5, 2), torch.int32, (1, 5))), dict(inv_freq=Dev((31,), F32)),
                dict(axis_pairs=(8, 25)), dict(q_weight=Dev((32,), F32)), dict(q_weight=Dev((64,), F16)),
                dict(pairs="both"), dict(q_out=Dev((2, 4, 5, 64), F16)), dict(q_out=Dev((2, 5, 4, 64), BF16)),
                dict(q_out=Dev((2, 5, 4, 64), F16, (0, 256, 64, 1))), dict(heads_first=True)):
        with pytest.raises(ValueError):
            binding.svdq_rope_axes(**rope_args(**bad))
    assert len(rec.calls) == 2


def test_statuses_under_address_and_undefined_behaviour_sanitizers():
    if not (os.path.exists("/opt/rocm/bin/hipcc") or shutil.which("hipcc")):
        pytest.skip("hipcc not available")
    from bit_w4a4_quantized_amd.build import BUILD_DIR, build_host_check
    exe = build_host_check(check="abi_check_block.cpp", exe=os.path.join(BUILD_DIR, "svdq_abi_check_block"))
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "OK: 0 failure(s)" in r.stdout, r.stdout


# ------------------------------------------------------------------ offline preparation
@pytest.mark.parametrize("types,qmax", [("int8", 127.0), ("e4m3", 448.0)])
def test_quantize_rows(types, qmax):
    """Codes times scale give the weight back within half a step; a row of zeros has codes 0 and a finite scale."""
    w = torch.randn(7, 40, generator=torch.Generator().manual_seed(4)) * 10.0 ** torch.arange(-3.0, 4.0)[:, None]
    w[2] = 0
    codes, scales = prepare.quantize_rows(w, types)
    assert codes.shape == w.shape and codes.is_contiguous() and scales.dtype == torch.float32
    assert bool(torch.isfinite(scales).all()) and not bool(codes[2].float().any())
    c = codes.double()
    assert float(c.abs().max()) == qmax
    back = c * scales.double()[:, None]
    step = 0.5 if types == "int8" else torch.clamp(c.abs() * 2.0 ** -4, min=2.0 ** -10)
    assert bool(((back - w.double()).abs() <= step * scales.double()[:, None] * 1.001 + w.double().abs() * 2.0 ** -20).all())


def test_rope_frequencies():
    f = prepare.rope_frequencies((8, 0, 3), 100.0)
    want = [100.0 ** (-j / 8) for j in range(8)] + [100.0 ** (-j / 3) for j in range(3)]
    assert f.dtype == torch.float32 and torch.allclose(f.double(), torch.tensor(want, dtype=torch.float64), rtol=2.0 ** -23)
