"""ctypes binding over libsvdq.so (the C ABI in include/svdq.h).

Argument marshalling only: every computation runs in the HIP kernels of the
library.  Tensors are torch tensors on the current HIP device (PyTorch is used
for device memory and streams); their data pointers and the current stream
are handed to the C entry points of the same names.  The module refuses to
run when the library is missing.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
# SVDQ_LIBRARY may name another build of the same library (same ABI), e.g. a tuning variant.
LIB_PATH = os.environ.get("SVDQ_LIBRARY") or os.path.join(HERE, "libsvdq.so")

FORMATS = {"int4": 0, "int8": 1, "fp4": 2, "int4_e2m3": 3, "mxfp4": 4}
GROUP = {"int4": 64, "int8": 64, "fp4": 16, "int4_e2m3": 64, "mxfp4": 32}
FMT_NAMES = {v: k for k, v in FORMATS.items()}

_lib = None

_c_int, _c_size, _vp = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
_c_i64, _c_float = ctypes.c_int64, ctypes.c_float


class RopeOperand(ctypes.Structure):
    """svdq_rope_operand."""
    _fields_ = [("inp", _vp), ("out", _vp), ("weight", _vp), ("heads", _c_int), ("in_batch", _c_i64),
                ("in_token", _c_i64), ("in_head", _c_i64), ("out_batch", _c_i64), ("out_token", _c_i64),
                ("out_head", _c_i64)]


_RopeOperands = RopeOperand * 2


class CacheStruct(ctypes.Structure):
    """svdq_paged_cache."""
    _fields_ = [("k", _vp), ("v", _vp), ("k_scales", _vp), ("v_scales", _vp), ("type", _c_int), ("pages", _c_i64),
                ("page_size", _c_int), ("heads", _c_int), ("dim", _c_int), ("page_stride", _c_i64),
                ("token_stride", _c_i64), ("head_stride", _c_i64), ("scale_page_stride", _c_i64),
                ("scale_token_stride", _c_i64), ("scale_head_stride", _c_i64)]


class BatchStruct(ctypes.Structure):
    """svdq_paged_batch."""
    _fields_ = [("page_table", _vp), ("table_stride", _c_i64), ("table_width", _c_int), ("starts", _vp), ("context", _vp),
                ("sequences", _c_int)]


_SIGS = {
    "svdq_code_row_bytes": (_c_size, [_c_int, _c_int]),
    "svdq_scale_row_bytes": (_c_size, [_c_int, _c_int]),
    "svdq_quantize_down": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _c_size, _vp]),
    "svdq_quantize_down_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "svdq_gemm_w4a4_up": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp]),
    "svdq_linear_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "svdq_linear": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _c_size, _vp, _vp]),
    "svdq_quantize_weight": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "svdq_pack_weight": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "svdq_linear_unfused_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "svdq_linear_unfused": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _c_size, _vp, _vp]),
    "svdq_gemm_w4a16": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _vp]),
    "svdq_gelu_tanh_smooth": (_c_int, [_vp, _vp, _c_int, _c_int, _vp, _vp]),
    "svdq_quantize_down_smooth": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp,
                                           _c_size, _vp]),
    "svdq_gemm_w4a4_up_gelu_smooth": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                               _c_int, _c_int, _vp, _vp]),
    "svdq_linear_folded": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                                    _vp, _c_size, _vp, _vp]),
    "svdq_relayout": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "svdq_linear_noalloc": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp]),
    "svdq_add_rmsnorm": (_c_int, [_vp, _c_i64, _c_int, _vp, _c_i64, _c_int, _vp, _c_int, _c_float, _c_int, _c_int,
                                  _c_int, _vp, _vp, _vp, _c_i64, _vp]),
    "svdq_gemm_act_residual": (_c_int, [_vp, _c_i64, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_int, _c_int, _c_int, _c_int,
                                        _c_int, _c_int, _vp, _c_i64, _vp, _c_size, _vp]),
    "svdq_gemm_act_residual_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "svdq_gemm_act_residual_kernel": (ctypes.c_char_p, [_c_int, _c_int, _c_int, _c_int, _c_size, _vp, _vp]),
    "svdq_rope_axes": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _c_int, _c_i64, _vp, _c_int, _vp,
                                _c_int, _c_float, _c_int, _vp]),
    "svdq_rope_append": (_c_int, [_vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_int, _c_int, _vp, _c_int, _vp, _c_int, _vp,
                                  _c_int, _c_float, _vp]),
    "svdq_tree_attention": (_c_int, [_vp, _vp, _vp, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_float, _vp, _c_i64, _c_int,
                                     _vp, _c_i64, _c_i64, _vp, _c_size, _vp]),
    "svdq_tree_attention_workspace_bytes": (_c_size, [_c_int] * 7),
    "svdq_cache_keep": (_c_int, [_vp, _vp, _vp, _c_i64, _c_int, _vp]),
    "svdq_status_string": (ctypes.c_char_p, [_c_int]),
    "svdq_version": (ctypes.c_char_p, []),
}


class SvdqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libsvdq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m bit_w4a4_quantized_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().svdq_status_string(s).decode()


def version() -> str:
    return lib().svdq_version().decode()


def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _p(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def _raw_stream_fn():
    """A cheap reader of the current stream's handle for a device index: torch's raw-stream
    accessor when it has one (no Stream object per call), else current_stream()."""
    import torch
    fn = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if fn is not None:
        return fn
    return lambda dev: torch.cuda.current_stream(dev).cuda_stream


def _new_on(stream, shape, dtype, device, returned=True):
    """torch.empty from the pool of `stream`, a handle: what a call writes there must not be a block
    that the current stream has freed and may still be using.  A returned tensor may be used and
    freed on the current stream, so the allocator learns of that stream too."""
    import torch
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(here)
    return t


def _new(stream, shape, dtype, device):
    """torch.empty where a call on `stream` (None: the current one) may write at once."""
    import torch
    return torch.empty(shape, dtype=dtype, device=device) if stream is None else _new_on(stream, shape, dtype, device)


def _new_workspace(stream, nbytes, device):
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if stream is None else \
        _new_on(stream, nbytes, torch.uint8, device, returned=False)


def _check(name: str, st: int):
    if st != 0:
        raise SvdqError(name, st)


def _need(t, dtype, shape, what):
    """A device tensor of this dtype and shape (None: any), contiguous; else ValueError.  The
    C ABI sees only pointers, so a wrong size would become an out-of-bounds device access:
    every tensor argument is checked here, before any launch."""
    if t is None:
        raise ValueError(f"{what} is required")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    if dtype is not None and t.dtype != dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


def _bytes_dtypes():
    """Code tensors are bytes: uint8, or int8 (e.g. INT8 codes as they were computed)."""
    import torch
    return (torch.uint8, torch.int8)


def _absent(t, what, why):
    if t is not None:
        raise ValueError(f"{what} must be None {why}")


def _check_kernel_b(xq, xs, t, wq, ws, l2, bias, K, fmt, y, lam_next=None):
    """Shapes of Kernel B's operands: (M, N, r).  r comes from l2 and must match t."""
    import torch
    if xq is None or wq is None:
        raise ValueError("xq and wq are required")
    M, N = code_rows(xq), code_rows(wq)
    r = 0 if l2 is None else int(l2.shape[0])
    f16 = torch.float16
    _need(xq, _bytes_dtypes(), code_shape(M, K, fmt), "xq")
    _need(xs, scale_dtype(fmt), scale_shape(M, K, fmt), "xs")
    _need(wq, _bytes_dtypes(), code_shape(N, K, fmt), "wq")
    _need(ws, scale_dtype(fmt), scale_shape(N, K, fmt), "ws")
    if r:
        _need(l2, f16, (r, N), "l2")
        _need(t, f16, (M, r), "t")
    else:
        _absent(t, "t", "when l2 is None (no branch)")
    if bias is not None:
        _need(bias, f16, (N,), "bias")
    if y is not None:
        _need(y, f16, (M, N), "y")
    if lam_next is not None:
        _need(lam_next, torch.float32, (N,), "lam_next")
    return M, N, r


def _check_weight(wq, ws, K, fmt):
    import torch
    if wq is None:
        raise ValueError("wq is required")
    N = code_rows(wq)
    _need(wq, _bytes_dtypes(), code_shape(N, K, fmt), "wq")
    _need(ws, scale_dtype(fmt), scale_shape(N, K, fmt), "ws")
    return N


def _check_branch(l1t, l2, K, N):
    """r from l1t [r, K] and l2 [r, N]: both present or both None."""
    import torch
    if (l1t is None) != (l2 is None):
        raise ValueError("l1t and l2 must both be given or both be None")
    if l1t is None:
        return 0
    r = int(l1t.shape[0])
    _need(l1t, torch.float16, (r, K), "l1t")
    _need(l2, torch.float16, (r, N), "l2")
    return r


# ------------------------------------------------------------------ sizes
@functools.lru_cache(maxsize=1024)
def code_row_bytes(K: int, fmt) -> int:
    return int(lib().svdq_code_row_bytes(K, _fmt(fmt)))


@functools.lru_cache(maxsize=4096)
def code_shape(rows: int, K: int, fmt):
    """Shape of a code tensor: chunk-major [K/64, rows, bytes per 64-K chunk] (32 for packed
    INT4, FP4 and MXFP4, 48 for the E2M3 container, 64 for INT8)."""
    name = fmt if isinstance(fmt, str) else FMT_NAMES[int(fmt)]
    return (K // 64, rows, {"int4": 32, "int4_e2m3": 48, "int8": 64, "fp4": 32, "mxfp4": 32}[name])


def code_rows(q) -> int:
    """Rows (tokens or output columns) of a code tensor in either layout."""
    return int(q.shape[1]) if q.dim() == 3 else int(q.shape[0])


def scale_row_entries(K: int, fmt) -> int:
    name = fmt if isinstance(fmt, str) else FMT_NAMES[int(fmt)]
    return K // GROUP[name]


@functools.lru_cache(maxsize=4096)
def scale_shape(rows: int, K: int, fmt):
    """Shape of the scale tensor: group-major [K/64, rows] for the INT formats; chunk-major
    [K/64, rows, 4] (FP4) or [K/64, rows, 2] (MXFP4)."""
    name = fmt if isinstance(fmt, str) else FMT_NAMES[int(fmt)]
    if name in ("int4", "int4_e2m3", "int8"):
        return (K // 64, rows)
    return (K // 64, rows, {"fp4": 4, "mxfp4": 2}[name])


def scale_dtype(fmt):
    import torch
    return torch.uint8 if _fmt(fmt) in (2, 4) else torch.float16   # E4M3 / E8M0 bytes


@functools.lru_cache(maxsize=4096)
def linear_workspace_bytes(M: int, K: int, r: int, fmt) -> int:
    return int(lib().svdq_linear_workspace_bytes(M, K, r, _fmt(fmt)))


@functools.lru_cache(maxsize=4096)
def linear_unfused_workspace_bytes(M: int, N: int, K: int, r: int, fmt) -> int:
    return int(lib().svdq_linear_unfused_workspace_bytes(M, N, K, r, _fmt(fmt)))


# ------------------------------------------------------------------ entry points (same names as the C ABI)
@functools.lru_cache(maxsize=4096)
def quantize_down_workspace_bytes(M: int, K: int, r: int, fmt) -> int:
    return int(lib().svdq_quantize_down_workspace_bytes(M, K, r, _fmt(fmt)))


def _outputs_kernel_a(M, K, r, fmt, dev, xq, xs, t, stream):
    """Kernel A's outputs: every given one is checked before any missing one is allocated."""
    import torch
    if xq is not None:
        _need(xq, _bytes_dtypes(), code_shape(M, K, fmt), "xq")
    if xs is not None:
        _need(xs, scale_dtype(fmt), scale_shape(M, K, fmt), "xs")
    if r:
        if t is not None:
            _need(t, torch.float16, (M, r), "t")
    else:
        _absent(t, "t", "when l1t is None (no branch)")
    if xq is None:
        xq = _new(stream, code_shape(M, K, fmt), torch.uint8, dev)
    if xs is None:
        xs = _new(stream, scale_shape(M, K, fmt), scale_dtype(fmt), dev)
    if r and t is None:
        t = _new(stream, (M, r), torch.float16, dev)
    return xq, xs, t


def _workspace_kernel_a(M, K, r, fmt, dev, workspace, no_workspace, stream):
    if no_workspace:
        return None, 0
    if workspace is None:
        nb = quantize_down_workspace_bytes(M, K, r, fmt)
        workspace = _new_workspace(stream, nb, dev) if nb else None
    else:
        _need(workspace, None, None, "workspace")
    return workspace, (0 if workspace is None else workspace.numel() * workspace.element_size())


def svdq_quantize_down(x_hat, l1t, fmt, xq=None, xs=None, t=None, workspace=None, no_workspace=False,
                       stream=None):
    """Kernel A.  x_hat fp16 [M, K]; l1t fp16 [r, K] or None.  Returns (xq, xs, t).
    workspace: uint8 device tensor for the sliced-K partial sums (allocated here when None);
    no_workspace=True passes NULL (K not sliced)."""
    import torch
    _need(x_hat, torch.float16, None, "x_hat")
    M, K = x_hat.shape
    r = 0 if l1t is None else int(l1t.shape[0])
    if l1t is not None:
        _need(l1t, torch.float16, (r, K), "l1t")
    dev = x_hat.device
    xq, xs, t = _outputs_kernel_a(M, K, r, fmt, dev, xq, xs, t, stream)
    workspace, ws_bytes = _workspace_kernel_a(M, K, r, fmt, dev, workspace, no_workspace, stream)
    _check("svdq_quantize_down", lib().svdq_quantize_down(
        _p(x_hat), _p(l1t), M, K, r, _fmt(fmt), _p(xq), _p(xs), _p(t), _p(workspace), ws_bytes,
        _stream(stream)))
    return xq, xs, t


def svdq_gemm_w4a4_up(xq, xs, t, wq, ws, l2, bias, K, fmt, y=None, stream=None):
    """Kernel B.  Returns y fp16 [M, N]."""
    import torch
    M, N, r = _check_kernel_b(xq, xs, t, wq, ws, l2, bias, K, fmt, y)
    if y is None:
        y = _new(stream, (M, N), torch.float16, xq.device)
    _check("svdq_gemm_w4a4_up", lib().svdq_gemm_w4a4_up(
        _p(xq), _p(xs), _p(t), _p(wq), _p(ws), _p(l2), _p(bias), M, N, K, r, _fmt(fmt), _p(y), _stream(stream)))
    return y


def _layer_args(x, l1t, wq, ws, l2, bias, fmt, y, workspace, stream, need_fn, what="x_hat"):
    """Checks of a whole-layer call's tensors; returns (M, N, K, r, y, workspace, bytes)."""
    import torch
    _need(x, torch.float16, None, what)
    M, K = x.shape
    N = _check_weight(wq, ws, K, fmt)
    r = _check_branch(l1t, l2, K, N)
    if bias is not None:
        _need(bias, torch.float16, (N,), "bias")
    if y is None:
        y = _new(stream, (M, N), torch.float16, x.device)
    else:
        _need(y, torch.float16, (M, N), "y")
    need = need_fn(M, N, K, r)
    if workspace is None:
        workspace = _new_workspace(stream, max(need, 16), x.device)
    else:
        _need(workspace, None, None, "workspace")
    return M, N, K, r, y, workspace, workspace.numel() * workspace.element_size()


def svdq_linear(x_hat, l1t, wq, ws, l2, bias, fmt, workspace=None, y=None, stream=None):
    """Kernel A then Kernel B.  Returns y fp16 [M, N]."""
    M, N, K, r, y, workspace, wb = _layer_args(x_hat, l1t, wq, ws, l2, bias, fmt, y, workspace, stream,
                                               lambda M, N, K, r: linear_workspace_bytes(M, K, r, fmt))
    _check("svdq_linear", lib().svdq_linear(
        _p(x_hat), _p(l1t), _p(wq), _p(ws), _p(l2), _p(bias), M, N, K, r, _fmt(fmt),
        _p(workspace), wb, _p(y), _stream(stream)))
    return y


def _outputs_weight(N, K, fmt, dev, wq, ws, stream):
    """The weight quantizer's outputs: every given one is checked before any missing one is
    allocated."""
    import torch
    if wq is not None:
        _need(wq, _bytes_dtypes(), code_shape(N, K, fmt), "wq")
    if ws is not None:
        _need(ws, scale_dtype(fmt), scale_shape(N, K, fmt), "ws")
    if wq is None:
        wq = _new(stream, code_shape(N, K, fmt), torch.uint8, dev)
    if ws is None:
        ws = _new(stream, scale_shape(N, K, fmt), scale_dtype(fmt), dev)
    return wq, ws


def svdq_quantize_weight(r_t, fmt, wq=None, ws=None, stream=None):
    """Offline: R^T fp32 [N, K] -> (wq, ws)."""
    import torch
    _need(r_t, torch.float32, None, "r_t")
    N, K = r_t.shape
    wq, ws = _outputs_weight(N, K, fmt, r_t.device, wq, ws, stream)
    _check("svdq_quantize_weight", lib().svdq_quantize_weight(
        _p(r_t), N, K, _fmt(fmt), _p(wq), _p(ws), _stream(stream)))
    return wq, ws


def svdq_pack_weight(codes, scales, fmt, wq=None, ws=None, stream=None):
    """Codes int8 [N, K] and fp16 scales [N, K/64] computed elsewhere (e.g. GPTQ) -> (wq, ws) in
    the layouts Kernel B reads (INT formats)."""
    import torch
    _need(codes, torch.int8, None, "codes")
    N, K = codes.shape
    _need(scales, torch.float16, (N, K // 64), "scales")
    wq, ws = _outputs_weight(N, K, fmt, codes.device, wq, ws, stream)
    _check("svdq_pack_weight", lib().svdq_pack_weight(_p(codes), _p(scales), N, K, _fmt(fmt), _p(wq), _p(ws),
                                                      _stream(stream)))
    return wq, ws


def svdq_linear_unfused(x_hat, l1t, wq, ws, l2, bias, fmt, workspace=None, y=None, stream=None):
    """The branch as separate kernels (measurement only).  Returns y fp16 [M, N]."""
    M, N, K, r, y, workspace, wb = _layer_args(
        x_hat, l1t, wq, ws, l2, bias, fmt, y, workspace, stream,
        lambda M, N, K, r: linear_unfused_workspace_bytes(M, N, K, r, fmt))
    _check("svdq_linear_unfused", lib().svdq_linear_unfused(
        _p(x_hat), _p(l1t), _p(wq), _p(ws), _p(l2), _p(bias), M, N, K, r, _fmt(fmt),
        _p(workspace), wb, _p(y), _stream(stream)))
    return y


def svdq_gemm_w4a16(x, wq, ws, bias, y=None, stream=None):
    """W4A16 control.  x fp16 [M, K]; wq, ws: SVDQ_INT4_G64 codes and scales of the N output
    columns (code_shape / scale_shape)."""
    import torch
    _need(x, torch.float16, None, "x")
    M, K = x.shape
    N = _check_weight(wq, ws, K, "int4")
    if bias is not None:
        _need(bias, torch.float16, (N,), "bias")
    if y is None:
        y = _new(stream, (M, N), torch.float16, x.device)
    else:
        _need(y, torch.float16, (M, N), "y")
    _check("svdq_gemm_w4a16", lib().svdq_gemm_w4a16(
        _p(x), _p(wq), _p(ws), _p(bias), M, N, K, _p(y), _stream(stream)))
    return y


def svdq_gelu_tanh_smooth(y, lam, out=None, stream=None):
    """fp16(gelu_tanh(y) / lam) for y fp16 [M, C], lam fp32 [C]."""
    import torch
    _need(y, torch.float16, None, "y")
    M, C = y.shape
    _need(lam, torch.float32, (C,), "lam")
    if out is None:
        out = _new(stream, (M, C), torch.float16, y.device)
    else:
        _need(out, torch.float16, (M, C), "out")
    _check("svdq_gelu_tanh_smooth", lib().svdq_gelu_tanh_smooth(
        _p(y), _p(lam), M, C, _p(out), _stream(stream)))
    return out


def svdq_quantize_down_smooth(x, lam, l1t, fmt, xq=None, xs=None, t=None, workspace=None, no_workspace=False,
                              stream=None):
    """Kernel A on unsmoothed x fp16 [M, K] with the layer's factors lam fp32 [K]:
    the codes, scales and T of X_hat = fp16(x / lam).  Returns (xq, xs, t).  Workspace as
    for svdq_quantize_down."""
    import torch
    _need(x, torch.float16, None, "x")
    M, K = x.shape
    r = 0 if l1t is None else int(l1t.shape[0])
    _need(lam, torch.float32, (K,), "lam")
    if l1t is not None:
        _need(l1t, torch.float16, (r, K), "l1t")
    dev = x.device
    xq, xs, t = _outputs_kernel_a(M, K, r, fmt, dev, xq, xs, t, stream)
    workspace, ws_bytes = _workspace_kernel_a(M, K, r, fmt, dev, workspace, no_workspace, stream)
    _check("svdq_quantize_down_smooth", lib().svdq_quantize_down_smooth(
        _p(x), _p(lam), _p(l1t), M, K, r, _fmt(fmt), _p(xq), _p(xs), _p(t), _p(workspace), ws_bytes,
        _stream(stream)))
    return xq, xs, t


def svdq_gemm_w4a4_up_gelu_smooth(xq, xs, t, wq, ws, l2, bias, lam_next, K, fmt, y=None, stream=None):
    """Kernel B with an MLP's glue in its epilogue: fp16(gelu(Y) / lam_next), lam_next fp32 [N]."""
    import torch
    if lam_next is None:
        raise ValueError("lam_next is required")
    M, N, r = _check_kernel_b(xq, xs, t, wq, ws, l2, bias, K, fmt, y, lam_next)
    if y is None:
        y = _new(stream, (M, N), torch.float16, xq.device)
    _check("svdq_gemm_w4a4_up_gelu_smooth", lib().svdq_gemm_w4a4_up_gelu_smooth(
        _p(xq), _p(xs), _p(t), _p(wq), _p(ws), _p(l2), _p(bias), _p(lam_next), M, N, K, r, _fmt(fmt), _p(y),
        _stream(stream)))
    return y


def svdq_linear_folded(x, lam_in, l1t, wq, ws, l2, bias, lam_next, fmt, workspace=None, y=None, stream=None):
    """The layer with either fold: lam_in fp32 [K] (x unsmoothed) and/or lam_next fp32 [N]
    (output fp16(gelu(Y) / lam_next)); None for a fold not taken.  Returns y fp16 [M, N]."""
    import torch
    M, N, K, r, y, workspace, wb = _layer_args(x, l1t, wq, ws, l2, bias, fmt, y, workspace, stream,
                                               lambda M, N, K, r: linear_workspace_bytes(M, K, r, fmt), "x")
    if lam_in is not None:
        _need(lam_in, torch.float32, (K,), "lam_in")
    if lam_next is not None:
        _need(lam_next, torch.float32, (N,), "lam_next")
    _check("svdq_linear_folded", lib().svdq_linear_folded(
        _p(x), _p(lam_in), _p(l1t), _p(wq), _p(ws), _p(l2), _p(bias), _p(lam_next), M, N, K, r, _fmt(fmt),
        _p(workspace), wb, _p(y), _stream(stream)))
    return y


def canonical_code_shape(rows: int, K: int, fmt):
    """Exchange layout of codes: [rows, K] for INT8, [rows, K/2] (two 4-bit codes a byte) otherwise."""
    return (rows, K if _fmt(fmt) == FORMATS["int8"] else K // 2)


def canonical_scale_shape(rows: int, K: int, fmt):
    name = fmt if isinstance(fmt, str) else FMT_NAMES[int(fmt)]
    return (rows, K // GROUP[name])


def svdq_relayout(codes, scales, K, fmt, to_canonical, codes_out=None, scales_out=None, stream=None):
    """Codes and scales between the exchange layout (row-major, see canonical_code_shape) and the
    format's device layout.  to_canonical=True: device -> exchange.  Returns (codes, scales)."""
    import torch
    if codes is None:
        raise ValueError("codes is required")
    if to_canonical:
        rows = code_rows(codes)
        src_c, src_s = code_shape(rows, K, fmt), scale_shape(rows, K, fmt)
        dst_c, dst_s = canonical_code_shape(rows, K, fmt), canonical_scale_shape(rows, K, fmt)
    else:
        rows = int(codes.shape[0])
        src_c, src_s = canonical_code_shape(rows, K, fmt), canonical_scale_shape(rows, K, fmt)
        dst_c, dst_s = code_shape(rows, K, fmt), scale_shape(rows, K, fmt)
    _need(codes, _bytes_dtypes(), src_c, "codes")
    _need(scales, scale_dtype(fmt), src_s, "scales")
    if codes_out is not None:
        _need(codes_out, _bytes_dtypes(), dst_c, "codes_out")
    if scales_out is not None:
        _need(scales_out, scale_dtype(fmt), dst_s, "scales_out")
    if codes_out is None:
        codes_out = _new(stream, dst_c, torch.uint8, codes.device)
    if scales_out is None:
        scales_out = _new(stream, dst_s, scale_dtype(fmt), codes.device)
    _check("svdq_relayout", lib().svdq_relayout(_p(codes), _p(scales), rows, K, _fmt(fmt), 1 if to_canonical else 0,
                                                _p(codes_out), _p(scales_out), _stream(stream)))
    return codes_out, scales_out


# ------------------------------------------------------------------ a block's operators between its linears
# These calls are short next to their host work, so the checks of the usual case are few Python
# operations and everything that depends on sizes alone is cached.
ACTIVATIONS = {"none": 0, "gelu": 1, "silu": 2}


class _Dtypes:
    """torch and what the block operators ask of it, looked up once."""

    def __init__(self):
        import torch
        self.torch = torch
        self.code = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2, torch.int8: 3, torch.float8_e4m3fn: 4}
        self.half = (torch.float16, torch.bfloat16)
        self.operand = (torch.int8, torch.float8_e4m3fn, torch.float16, torch.bfloat16)
        self.f32 = (torch.float32,)
        self.raw_stream = _raw_stream_fn()


_dtypes = None


def _d():
    global _dtypes
    if _dtypes is None:
        _dtypes = _Dtypes()
    return _dtypes


def _rows(t, dtypes, shape, what):
    """The row stride of a 2-D device tensor whose rows are contiguous (any row stride that keeps
    them apart); else ValueError.  dtypes: those it may have."""
    if t is None:
        raise ValueError(f"{what} is required")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{what} must be one of {dtypes}, got {t.dtype}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{what} must have shape {shape or '[rows, columns]'}, got {tuple(t.shape)}")
    rows, cols = t.shape
    step, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{what}'s rows must be contiguous")
    if rows <= 1 or cols == 0:
        return cols
    if step < cols:
        raise ValueError(f"{what}'s rows must not overlap")
    return step


def _vector(t, dtypes, n, what):
    if t is None:
        raise ValueError(f"{what} is required")
    if not t.is_cuda or t.dtype not in dtypes or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous device tensor of shape ({n},) and one of {dtypes}, "
                         f"got {tuple(t.shape)} {t.dtype}")


def _launch(fn, args, tensors, stream):
    """One C call on the device of the tensors, the caller's: on `stream` when given, else on that
    device's current stream."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"all tensors must be on one device, got {tensors[0].device} and {t.device}")
    d = _dtypes
    torch = d.torch
    if dev == torch._C._cuda_getDevice():
        st = getattr(lib(), fn)(*args, d.raw_stream(dev) if stream is None else stream)
    else:
        with torch.cuda.device(dev):
            st = getattr(lib(), fn)(*args, d.raw_stream(dev) if stream is None else stream)
    if st != 0:
        raise SvdqError(fn, st)


def svdq_add_rmsnorm(x, weight, eps=1e-6, residual=None, out_format="int8", out=None, scales=None,
                     residual_out=None, stream=None):
    """RMS norm of x [M, K] (fp16 or bf16, rows any stride apart) plus a residual (x's type or
    fp32), weight [K] (x's type or fp32).  out_format "int8" or "e4m3": codes [M, K] and fp32
    scales [M], code * scale being the normed value; "same": [M, K] in x's type, no scales.
    Returns (out, scales, stream): stream = x + residual in the residual's type, None without one.
    residual_out may be residual, or x where the types agree."""
    d = _dtypes or _d()
    torch, code = d.torch, d.code
    xs = _rows(x, d.half, None, "x")
    shape = x.shape
    M, K = shape
    xd = x.dtype
    _vector(weight, (xd, torch.float32), K, "weight")
    if out_format == "int8":
        od = torch.int8
    elif out_format == "e4m3":
        od = torch.float8_e4m3fn
    elif out_format == "same":
        od = xd
        _absent(scales, "scales", "for a 16-bit output")
    else:
        raise ValueError(f"out_format must be 'int8', 'e4m3' or 'same', got {out_format!r}")
    rs = ros = rt = 0
    if residual is not None:
        rs, rt = _rows(residual, (xd, torch.float32), shape, "residual"), code[residual.dtype]
        if residual_out is not None:
            ros = _rows(residual_out, (residual.dtype,), shape, "residual_out")
    elif residual_out is not None:
        _absent(residual_out, "residual_out", "without a residual")
    if out is not None:
        _need(out, od, shape, "out")
    if scales is not None:
        _need(scales, torch.float32, (M,), "scales")
    given = (x, weight, residual, out, scales, residual_out)
    new = torch.empty if stream is None else functools.partial(_new_on, stream)
    if out is None:
        out = new(shape, dtype=od, device=x.device)
    if scales is None and od is not xd:
        scales = new((M,), dtype=torch.float32, device=x.device)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(residual) if rs == K and stream is None else \
            new(shape, dtype=residual.dtype, device=x.device)
        ros = K
    _launch("svdq_add_rmsnorm",
            (x.data_ptr(), xs, code[xd], _p(residual), rs, rt, weight.data_ptr(), code[weight.dtype], eps, M, K,
             code[od], out.data_ptr(), _p(scales), _p(residual_out), ros), given, stream)
    return out, scales, residual_out


@functools.lru_cache(maxsize=4096)
def gemm_act_residual_workspace_bytes(M: int, N: int, K: int, type_code: int) -> int:
    return int(lib().svdq_gemm_act_residual_workspace_bytes(M, N, K, type_code))


def gemm_act_residual_kernel(M: int, N: int, K: int, type_code: int, workspace_bytes=None):
    """(kernel, splits, tail) that svdq_gemm_act_residual takes for these sizes, with the workspace it
    asks for when None; see include/svdq.h."""
    if workspace_bytes is None:
        workspace_bytes = gemm_act_residual_workspace_bytes(M, N, K, type_code)
    splits, tail = ctypes.c_int(0), ctypes.c_int(0)
    name = lib().svdq_gemm_act_residual_kernel(M, N, K, type_code, workspace_bytes, ctypes.addressof(splits),
                                               ctypes.addressof(tail))
    return None if name is None else (name.decode(), splits.value, tail.value)


def svdq_gemm_act_residual(x, w, xs=None, ws=None, bias=None, activation="none", residual=None, out_dtype=None,
                           y=None, workspace=None, stream=None):
    """y = act((x w^T) * xs[:, None] * ws + bias) + residual, rounded once.  x [M, K] and w [N, K]
    int8, float8_e4m3fn, fp16 or bf16 (x's rows any stride apart); xs [M], ws [N] fp32; bias [N],
    residual and y [M, N] of out_dtype (fp16 or bf16; x's type, or fp16 for 8-bit x, when None);
    activation "none", "gelu" (tanh) or "silu".  y may be residual.  workspace: device bytes for
    the sums of K's splits (gemm_act_residual_workspace_bytes; allocated here when None)."""
    d = _dtypes or _d()
    torch, code = d.torch, d.code
    xt = _rows(x, d.operand, None, "x")
    M, K = x.shape
    dtype = x.dtype
    if w is None or w.dim() != 2:
        raise ValueError("w must be a device tensor [N, K]")
    N = w.shape[0]
    _need(w, dtype, (N, K), "w")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {tuple(ACTIVATIONS)}, got {activation!r}")
    if out_dtype is None:
        out_dtype = dtype if dtype in d.half else torch.float16
    elif out_dtype not in d.half:
        raise ValueError(f"out_dtype must be float16 or bfloat16, got {out_dtype}")
    if xs is not None:
        _vector(xs, d.f32, M, "xs")
    if ws is not None:
        _vector(ws, d.f32, N, "ws")
    if bias is not None:
        _vector(bias, (out_dtype,), N, "bias")
    rs = 0 if residual is None else _rows(residual, (out_dtype,), (M, N), "residual")
    given = (x, w, xs, ws, bias, residual, y, workspace)
    if workspace is not None:
        _need(workspace, None, None, "workspace")
        room = workspace.numel() * workspace.element_size()
    else:
        room = gemm_act_residual_workspace_bytes(M, N, K, code[dtype])
        if room:
            workspace = _new_workspace(stream, room, x.device)
    if y is not None:
        yt = _rows(y, (out_dtype,), (M, N), "y")
    else:
        y = _new(stream, (M, N), out_dtype, x.device)
        yt = N
    _launch("svdq_gemm_act_residual",
            (x.data_ptr(), xt, _p(xs), w.data_ptr(), _p(ws), _p(bias), _p(residual), rs, M, N, K, code[dtype], act,
             code[out_dtype], y.data_ptr(), yt, _p(workspace), room), given, stream)
    return y


def _heads_layout(size, step, heads_first, what):
    """Sizes and (batch, token, head) strides of [batch, tokens, heads, dim] (heads_first: [batch,
    heads, tokens, dim]), or of the same without the batch."""
    if len(size) not in (3, 4):
        raise ValueError(f"{what} must have 3 or 4 dimensions, got {len(size)}")
    if step[-1] != 1 and size[-1] > 1:
        raise ValueError(f"{what}'s heads must be contiguous")
    if len(size) == 3:
        size, step = (1, *size), (0, *step)
    if heads_first:
        size, step = (size[0], size[2], size[1], size[3]), (step[0], step[2], step[1])
    return tuple(size), tuple(step[:3])


@functools.lru_cache(maxsize=1024)
def _rope_plan(q, k, q_out, k_out, positions, axis_pairs, heads_first):
    """What svdq_rope_axes checks and works out from sizes alone.  Operands as (shape, strides) or
    None; returns the operands without their pointers, (B, T, D), P, the axes' array, the positions'
    batch stride and the shapes of outputs to allocate."""
    ops, shapes, sizes = _RopeOperands(), [None, None], None
    for i, (name, x, out) in enumerate((("q", q, q_out), ("k", k, k_out))):
        if x is None:
            continue
        size, step = _heads_layout(*x, False, name)
        if sizes is None:
            sizes = size
        elif (size[0], size[1], size[3]) != (sizes[0], sizes[1], sizes[3]) or len(x[0]) != len(q[0]):
            raise ValueError(f"k must have q's batch, tokens and dim, got {tuple(x[0])} and {tuple(q[0])}")
        if out is None:
            s = tuple(x[0])
            shapes[i] = (*s[:-3], s[-2], s[-3], s[-1]) if heads_first else s
            steps = [1]
            for n in reversed(shapes[i][1:]):
                steps.insert(0, steps[0] * n)
            out = (shapes[i], tuple(steps))
        if len(out[0]) != len(x[0]):
            raise ValueError(f"{name}_out must have {len(x[0])} dimensions")
        osize, ostep = _heads_layout(*out, heads_first, name + "_out")
        if osize != size:
            raise ValueError(f"{name}_out must have {name}'s sizes in the output's layout, got {tuple(out[0])}")
        if any(n > 1 and s < 1 for n, s in zip(osize, ostep)):
            raise ValueError(f"{name}_out must not overlap itself")
        ops[i] = RopeOperand(0, 0, 0, size[2], *step, *ostep)
    B, T, _, D = sizes
    axes = len(axis_pairs)
    if tuple(positions) == (T, axes):
        pos_batch = 0
    elif len(q[0]) == 4 and tuple(positions) == (B, T, axes):
        pos_batch = T * axes
    else:
        raise ValueError(f"positions must have shape ({T}, {axes}) or ({B}, {T}, {axes}), got {tuple(positions)}")
    return bytes(ops), (B, T, D), sum(axis_pairs), (_c_int * axes)(*axis_pairs), pos_batch, shapes


def _rope_out(x, shape, stream):
    if stream is not None:
        return _new_on(stream, shape, x.dtype, x.device)
    return _dtypes.torch.empty_like(x) if shape == x.shape and x.is_contiguous() else x.new_empty(shape)


def svdq_rope_axes(q, k, positions, inv_freq, axis_pairs, pairs="adjacent", q_weight=None, k_weight=None, eps=1e-6,
                   inverse=False, heads_first=False, q_out=None, k_out=None, stream=None):
    """Rotary positions with several axes on q [batch, tokens, heads, dim] and k (the same with its
    own number of heads; None for q alone), fp16 or bf16, or both without the batch; any strides
    with contiguous heads.  positions [tokens, axes] or [batch, tokens, axes] int32 or fp32;
    inv_freq fp32 [P]; axis_pairs: pairs that turn by each axis, P in all, 2 P <= dim.  pairs:
    "adjacent" (2p, 2p + 1) or "halves" (p, p + P).  q_weight, k_weight fp32 [dim]: the heads' RMS
    norm in front.  inverse: turn back (the gradient).  Outputs [batch, tokens, heads, dim], or
    [batch, heads, tokens, dim] with heads_first; q_out may be q, k_out k, with heads_first False.
    Returns (q_out, k_out)."""
    d = _dtypes or _d()
    torch = d.torch
    if q is None:
        raise ValueError("q is required")
    if pairs not in ("adjacent", "halves"):
        raise ValueError(f"pairs must be 'adjacent' or 'halves', got {pairs!r}")
    dtype = q.dtype
    if dtype not in d.half:
        raise ValueError(f"q must be float16 or bfloat16, got {dtype}")
    if k is None:
        _absent(k_weight, "k_weight", "without k")
        _absent(k_out, "k_out", "without k")
    for name, t in (("q", q), ("k", k), ("q_out", q_out), ("k_out", k_out)):
        if t is not None and not (t.is_cuda and t.dtype == dtype):
            raise ValueError(f"{name} must be a {dtype} device tensor")
    if positions is None or not positions.is_cuda or positions.dtype not in (torch.int32, torch.float32) or not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int32 or float32 device tensor")
    layout = lambda t: None if t is None else (t.shape, t.stride())  # noqa: E731
    axis_pairs = tuple(axis_pairs)
    blank, (B, T, D), P, axes, pos_batch, shapes = _rope_plan(
        layout(q), layout(k), layout(q_out), layout(k_out), positions.shape, axis_pairs, bool(heads_first))
    _vector(inv_freq, d.f32, P, "inv_freq")
    ops = _RopeOperands.from_buffer_copy(blank)
    given = (q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out)
    if q_weight is not None:
        _vector(q_weight, d.f32, D, "q_weight")
        ops[0].weight = q_weight.data_ptr()
    if q_out is None:
        q_out = _rope_out(q, shapes[0], stream)
    ops[0].inp, ops[0].out = q.data_ptr(), q_out.data_ptr()
    if k is not None:
        if k_weight is not None:
            _vector(k_weight, d.f32, D, "k_weight")
            ops[1].weight = k_weight.data_ptr()
        if k_out is None:
            k_out = _rope_out(k, shapes[1], stream)
        ops[1].inp, ops[1].out = k.data_ptr(), k_out.data_ptr()
    _launch("svdq_rope_axes",
            (ctypes.addressof(ops), 1 if k is None else 2, B, T, D, d.code[dtype], positions.data_ptr(),
             1 if positions.dtype == torch.float32 else 0, pos_batch, inv_freq.data_ptr(), len(axis_pairs), axes,
             1 if pairs == "halves" else 0, eps, 1 if inverse else 0),
            given, stream)
    return q_out, k_out


# ------------------------------------------------------------------ a paged cache of keys and values
def _apart(shape, stride, what):
    """The strides of a tensor's dimensions, 0 for those of one element or none; ValueError where elements share
    memory."""
    step = tuple(0 if n <= 1 else s for n, s in zip(shape, stride))
    reach = 1
    for s, n in sorted((s, n) for s, n in zip(step, shape) if n > 1):
        if s < reach:
            raise ValueError(f"{what} must not overlap itself")
        reach = s * (n - 1) + reach
    return step


class PagedCache:
    """The pages of a cache, checked once: keys k and values v [pages, page_size, heads, dim] of one type (fp16 or
    bf16, or int8 or float8_e4m3fn codes) and one layout (any strides, multiples of 16 bytes, with contiguous
    heads; e.g. a transposed view of pages that keep heads first), and for codes the fp32 scales [pages,
    page_size, heads] of both, a head's value being code * scale.  page_size: a power of two; dim: a multiple of
    8 (of 16 for codes) up to 256.  The operators read and write the tensors in place; the handle keeps
    references to them.  A captured graph holds the tensors' addresses, not this object's."""

    def __init__(self, k, v, k_scales=None, v_scales=None):
        d = _dtypes or _d()
        for name, t in (("k", k), ("v", v)):
            if t is None:
                raise ValueError(f"{name} is required")
            if not t.is_cuda or t.dtype not in d.operand:
                raise ValueError(f"{name} must be a device tensor and one of {d.operand}, got {t.dtype}")
            if t.dim() != 4:
                raise ValueError(f"{name} must have shape [pages, page_size, heads, dim], got {tuple(t.shape)}")
        if v.dtype != k.dtype or v.shape != k.shape:
            raise ValueError(f"v must have k's type and shape, got {v.dtype} {tuple(v.shape)}")
        pages, size, heads, dim = k.shape
        if size < 1 or size & (size - 1) or size > 1 << 16:
            raise ValueError(f"page_size must be a power of two up to {1 << 16}, got {size}")
        each = 8 if k.dtype in d.half else 16
        if not 8 <= dim <= 256 or dim % each or heads < 1:
            raise ValueError(f"a head of {k.dtype} must have a multiple of {each} values up to 256, got {dim} ({heads} heads)")
        steps = [_apart(t.shape, t.stride(), name) for name, t in (("k", k), ("v", v))]
        if any(t.stride()[3] != 1 for t in (k, v)):
            raise ValueError("the heads of k and v must be contiguous")
        if steps[0] != steps[1]:
            raise ValueError(f"k and v must have the same strides, got {k.stride()} and {v.stride()}")
        if any(s % each for s in steps[0][:3]) or k.data_ptr() % 16 or v.data_ptr() % 16:
            raise ValueError("the strides and addresses of k and v must be multiples of 16 bytes")
        scale_step = (0, 0, 0)
        if k.dtype in d.half:
            _absent(k_scales, "k_scales", "for a 16-bit cache")
            _absent(v_scales, "v_scales", "for a 16-bit cache")
        else:
            for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
                if t is None:
                    raise ValueError(f"{name} is required for a cache of codes")
                if not t.is_cuda or t.dtype != d.torch.float32 or t.shape != k.shape[:3]:
                    raise ValueError(f"{name} must be a float32 device tensor of shape {tuple(k.shape[:3])}")
            scale_steps = [_apart(t.shape, t.stride(), name) for name, t in (("k_scales", k_scales), ("v_scales", v_scales))]
            if scale_steps[0] != scale_steps[1]:
                raise ValueError("k_scales and v_scales must have the same strides")
            scale_step = scale_steps[0]
        for t in (v, k_scales, v_scales):
            if t is not None and t.get_device() != k.get_device():
                raise ValueError("all tensors of a cache must be on one device")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.pages, self.page_size, self.heads, self.dim, self.dtype = pages, size, heads, dim, k.dtype
        self.step_types = (k.dtype,) if k.dtype in d.half else d.half
        self._struct = CacheStruct(k.data_ptr(), v.data_ptr(), _p(k_scales), _p(v_scales), d.code[k.dtype], pages, size,
                                   heads, dim, *steps[0][:3], *scale_step)
        self._at = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, pages, page_size, heads, dim, dtype, device="cuda"):
        """A cache of new pages, zeroed (what attention does not see may hold anything)."""
        import torch
        shape = (pages, page_size, heads, dim)
        new = lambda: torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) if dtype.itemsize == 1 else \
            torch.zeros(shape, dtype=dtype, device=device)  # noqa: E731
        scale = lambda: torch.zeros(shape[:3], device=device) if dtype.itemsize == 1 else None  # noqa: E731
        return cls(new(), new(), scale(), scale())


class PagedBatch:
    """A step's sequences, checked once and shared by the step's layers: page_table int32 [sequences, width] (slot s
    of a sequence is token s % page_size of page page_table[s // page_size]; an entry that is no page, e.g. -1, holds
    nothing), starts int32 [sequences + 1] (sequence b has the step's tokens starts[b] ... starts[b + 1] - 1) and
    context int32 [sequences] (tokens in the cache before the step).  The handle keeps references to the tensors;
    their contents may change between calls."""

    def __init__(self, page_table, starts, context):
        d = _dtypes or _d()
        i32 = (d.torch.int32,)
        step = _rows(page_table, i32, None, "page_table")
        n, width = page_table.shape
        _vector(starts, i32, n + 1, "starts")
        _vector(context, i32, n, "context")
        for t in (starts, context):
            if t.get_device() != page_table.get_device():
                raise ValueError("all tensors of a batch must be on one device")
        self.page_table, self.starts, self.context, self.sequences, self.width = page_table, starts, context, n, width
        self._struct = BatchStruct(page_table.data_ptr(), step, width, starts.data_ptr(), context.data_ptr(), n)
        self._at = ctypes.addressof(self._struct)


def _paged(cache, batch):
    if not isinstance(cache, PagedCache) or not isinstance(batch, PagedBatch):
        raise ValueError("cache must be a PagedCache and batch a PagedBatch")


@functools.lru_cache(maxsize=1024)
def _append_plan(q, k, v, q_out, positions, axis_pairs, heads, dim):
    """What svdq_rope_append checks and works out from sizes alone: operands as (shape, strides), q None for none.
    Returns the operands without their pointers, tokens, P, the axes' array and the strides of v."""
    ops = _RopeOperands()
    tokens = k[0][0] if len(k[0]) == 3 else -1
    for name, x in (("k", k), ("v", v), ("q", q), ("q_out", q_out)):
        if x is None:
            continue
        shape, step = x
        want = (tokens, heads, dim) if name in "kv" else None
        if len(shape) != 3 or (want and tuple(shape) != want) or shape[0] != tokens or shape[2] != dim:
            raise ValueError(f"{name} must have shape [tokens, {heads if want else 'heads'}, {dim}], got {tuple(shape)}")
        if step[2] != 1:
            raise ValueError(f"{name}'s heads must be contiguous")
    if q is not None:
        if q[0][1] < 1:
            raise ValueError("q must have a head")
        out = q_out or (q[0], (q[0][1] * dim, dim, 1))
        if tuple(out[0]) != tuple(q[0]):
            raise ValueError(f"q_out must have q's shape, got {tuple(out[0])}")
        _apart(out[0], out[1], "q_out")
        ops[0] = RopeOperand(0, 0, 0, q[0][1], 0, *q[1][:2], 0, *out[1][:2])
    ops[1] = RopeOperand(0, 0, 0, heads, 0, *k[1][:2], 0, 0, 0)
    axes = len(axis_pairs)
    if tuple(positions) != (tokens, axes):
        raise ValueError(f"positions must have shape ({tokens}, {axes}), got {tuple(positions)}")
    return bytes(ops), tokens, sum(axis_pairs), (_c_int * axes)(*axis_pairs), v[1][:2]


_OPERAND_BYTES = ctypes.sizeof(RopeOperand)


def svdq_rope_append(cache, batch, q, k, v, positions, inv_freq, axis_pairs, pairs="adjacent", q_weight=None,
                     k_weight=None, eps=1e-6, q_out=None, stream=None):
    """A step's tokens into a paged cache, with the rotary positions of svdq_rope_axes on queries and keys.  q
    [tokens, heads, dim] (None for no queries), k and v [tokens, cache heads, dim], fp16 or bf16 (a 16-bit cache's
    own type); any strides with contiguous heads.  positions [tokens, axes] int32 or fp32; inv_freq fp32 [P],
    axis_pairs, pairs, q_weight, k_weight and eps as for svdq_rope_axes.  Keys and values go to the slots behind
    their sequence's context, quantized for a cache of codes (a scale per token and head).  Returns the turned
    queries [tokens, heads, dim] (q_out, which may be q)."""
    d = _dtypes or _d()
    torch = d.torch
    _paged(cache, batch)
    if k is None or v is None:
        raise ValueError("k and v are required")
    dtype = k.dtype
    if dtype not in cache.step_types:
        raise ValueError(f"k must be one of {cache.step_types} for a cache of {cache.dtype}, got {dtype}")
    if q is None:
        _absent(q_weight, "q_weight", "without q")
        _absent(q_out, "q_out", "without q")
    for name, t in (("k", k), ("v", v), ("q", q), ("q_out", q_out)):
        if t is not None and not (t.is_cuda and t.dtype == dtype):
            raise ValueError(f"{name} must be a {dtype} device tensor")
    if pairs not in ("adjacent", "halves"):
        raise ValueError(f"pairs must be 'adjacent' or 'halves', got {pairs!r}")
    if positions is None or not positions.is_cuda or positions.dtype not in (torch.int32, torch.float32) or not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int32 or float32 device tensor")
    axis_pairs = tuple(axis_pairs)
    blank, tokens, P, axes, v_step = _append_plan(
        None if q is None else (q.shape, q.stride()), (k.shape, k.stride()), (v.shape, v.stride()),
        None if q_out is None else (q_out.shape, q_out.stride()), positions.shape, axis_pairs, cache.heads, cache.dim)
    _vector(inv_freq, d.f32, P, "inv_freq")
    ops = _RopeOperands.from_buffer_copy(blank)
    given = (cache.k, batch.page_table, k, v, q, positions, inv_freq, q_weight, k_weight, q_out)
    ops[1].inp = k.data_ptr()
    if k_weight is not None:
        _vector(k_weight, d.f32, cache.dim, "k_weight")
        ops[1].weight = k_weight.data_ptr()
    at = ctypes.addressof(ops)
    if q is not None:
        if q_weight is not None:
            _vector(q_weight, d.f32, cache.dim, "q_weight")
            ops[0].weight = q_weight.data_ptr()
        if q_out is None:
            q_out = _rope_out(q, q.shape, stream)
        ops[0].inp, ops[0].out = q.data_ptr(), q_out.data_ptr()
    _launch("svdq_rope_append",
            (cache._at, batch._at, None if q is None else at, at + _OPERAND_BYTES, v.data_ptr(), *v_step, tokens,
             d.code[dtype], positions.data_ptr(), 1 if positions.dtype == torch.float32 else 0, inv_freq.data_ptr(),
             len(axis_pairs), axes, 1 if pairs == "halves" else 0, eps), given, stream)
    return q_out


@functools.lru_cache(maxsize=4096)
def tree_attention_workspace_bytes(sequences: int, tokens: int, heads: int, kv_heads: int, dim: int, table_width: int,
                                   page_size: int) -> int:
    return int(lib().svdq_tree_attention_workspace_bytes(sequences, tokens, heads, kv_heads, dim, table_width, page_size))


def svdq_tree_attention(cache, batch, q, tree=None, scale=None, out=None, workspace=None, stream=None):
    """Attention of a step's queries q [tokens, heads, dim] (fp16 or bf16; any strides with contiguous heads; turned
    as by svdq_rope_append) over their sequences' cached keys and values, the step's own among them.  Every token
    sees its sequence's context; of the step's tokens it sees those that its row of tree marks (bool or uint8
    [tokens, width]: column j is the sequence's j-th token of the step, columns past the width are not seen), or,
    without a tree, those up to itself: one decoded token, or a chunk of a prompt.  heads: a multiple of the
    cache's.  scale: dim ** -0.5 when None.  A row that sees nothing is zeros; tokens of no sequence keep what out
    held.  out may be q.  workspace: device bytes for the sums of the keys' parts (tree_attention_workspace_bytes;
    allocated here when None)."""
    d = _dtypes or _d()
    torch = d.torch
    _paged(cache, batch)
    if q is None:
        raise ValueError("q is required")
    dtype = q.dtype
    if dtype not in cache.step_types or not q.is_cuda:
        raise ValueError(f"q must be a device tensor and one of {cache.step_types} for a cache of {cache.dtype}, got {dtype}")
    if q.dim() != 3 or q.shape[2] != cache.dim:
        raise ValueError(f"q must have shape [tokens, heads, {cache.dim}], got {tuple(q.shape)}")
    tokens, heads, dim = q.shape
    if heads < 1 or heads % cache.heads:
        raise ValueError(f"q's heads must be a multiple of the cache's {cache.heads}, got {heads}")
    q_step = q.stride()
    if q_step[2] != 1:
        raise ValueError("q's heads must be contiguous")
    if scale is None:
        scale = dim ** -0.5
    t_step = t_width = 0
    at = None
    if tree is not None:
        t_step = _rows(tree, (torch.bool, torch.uint8), None, "tree")
        if tree.shape[0] != tokens:
            raise ValueError(f"tree must have a row for each of the {tokens} tokens, got {tree.shape[0]}")
        t_width = tree.shape[1]
        at = tree.data_ptr() or q.data_ptr()       # a tree without columns has no memory, and is a tree all the same
    if out is None:
        o_step = (heads * dim, dim)
    else:
        if not out.is_cuda or out.dtype != dtype or out.shape != q.shape or out.stride()[2] != 1:
            raise ValueError(f"out must be a {dtype} device tensor of shape {tuple(q.shape)} with contiguous heads")
        _apart(out.shape, out.stride(), "out")
        o_step = out.stride()
    given = (cache.k, batch.page_table, q, tree, out, workspace)
    if workspace is not None:
        _need(workspace, None, None, "workspace")
        room = workspace.numel() * workspace.element_size()
    else:
        room = tree_attention_workspace_bytes(batch.sequences, tokens, heads, cache.heads, dim, batch.width, cache.page_size)
        if room:
            workspace = _new_workspace(stream, room, q.device)
    if out is None:
        out = _rope_out(q, q.shape, stream)
    _launch("svdq_tree_attention",
            (cache._at, batch._at, q.data_ptr(), q_step[0], q_step[1], heads, tokens, d.code[dtype], scale, at, t_step,
             t_width, out.data_ptr(), o_step[0], o_step[1], _p(workspace), room), given, stream)
    return out


def svdq_cache_keep(cache, batch, path, stream=None):
    """Keeps a draft's accepted tokens: slot context + i of sequence b takes keys, values and scales of slot context
    + path[b, i], for path int32 [sequences, width] whose rows rise and end in negative entries.  batch: that of
    the step which drafted them (its context before the draft)."""
    d = _dtypes or _d()
    _paged(cache, batch)
    step = _rows(path, (d.torch.int32,), None, "path")
    if path.shape[0] != batch.sequences:
        raise ValueError(f"path must have a row for each of the {batch.sequences} sequences, got {path.shape[0]}")
    _launch("svdq_cache_keep", (cache._at, batch._at, path.data_ptr(), step, path.shape[1]),
            (cache.k, batch.page_table, path), stream)


# svdq_linear_noalloc's static device scratch (SVDQ_STATIC_SCRATCH_BYTES in include/svdq.h)
STATIC_SCRATCH_BYTES = 64 << 20


def svdq_linear_noalloc(x_hat, l1t, wq, ws, l2, bias, fmt, y, stream=None):
    """The fused layer with its intermediates in the library's static per-device scratch: no
    device allocation in the library, and none here either (the output y fp16 [M, N] is the
    caller's).  Calls that overlap on one GPU race on the scratch."""
    import torch
    if y is None:
        raise ValueError("y is required (this entry point allocates nothing)")
    _need(x_hat, torch.float16, None, "x_hat")
    M, K = x_hat.shape
    N = _check_weight(wq, ws, K, fmt)
    r = _check_branch(l1t, l2, K, N)
    if bias is not None:
        _need(bias, torch.float16, (N,), "bias")
    _need(y, torch.float16, (M, N), "y")
    _check("svdq_linear_noalloc", lib().svdq_linear_noalloc(
        _p(x_hat), _p(l1t), _p(wq), _p(ws), _p(l2), _p(bias), M, N, K, r, _fmt(fmt), _p(y), _stream(stream)))
    return y


class SvdqLinear:
    """The fused layer prepared for repeated calls (a serving loop, a benchmark's eager steps).

    The weight-side tensors -- residual codes and scales, L1^T, L2, bias -- are checked once
    here and their pointers kept (with references that keep the tensors alive); each call then
    checks only its activations and output, reuses a workspace kept for each stream and its largest M, and
    makes one svdq_linear call: the same kernels and results as svdq_linear, with a fraction of
    its per-call host work.  One thread at a time calls it.
    """

    def __init__(self, wq, ws, l1t, l2, bias, K: int, fmt):
        import torch
        self.K, self.fmt, self._F = int(K), fmt, _fmt(fmt)
        self.N = _check_weight(wq, ws, K, fmt)
        self.r = _check_branch(l1t, l2, K, self.N)
        if bias is not None:
            _need(bias, torch.float16, (self.N,), "bias")
        self._keep = (wq, ws, l1t, l2, bias)
        self._ptrs = (_p(l1t), _p(wq), _p(ws), _p(l2), _p(bias))
        self.device = wq.device
        self._dev_index = wq.device.index if wq.device.index is not None else torch.cuda.current_device()
        self._f16 = torch.float16
        self._kept = {}                      # of each stream's handle: (workspace, its bytes, rows it holds)
        self._ws_bytes, self._on = 0, (0, None)
        self._fn = lib().svdq_linear
        self._raw_stream = _raw_stream_fn()

    def _workspace(self, M: int):
        """The workspace of the call's stream, self._on: its handle, and the caller's `stream`."""
        handle, stream = self._on
        kept = self._kept.get(handle)
        if kept is None or M > kept[2]:
            nb = max(linear_workspace_bytes(M, self.K, self.r, self.fmt), 16)
            kept = self._kept[handle] = (_new_workspace(stream, nb, self.device), nb, M)
        self._ws_bytes = kept[1]
        return kept[0]

    def __call__(self, x_hat, y=None, stream=None):
        """x_hat fp16 [M, K] (smoothed) -> y fp16 [M, N] (allocated when None)."""
        if not (x_hat.is_cuda and x_hat.dtype == self._f16 and x_hat.dim() == 2 and x_hat.shape[1] == self.K
                and x_hat.is_contiguous()):
            _need(x_hat, self._f16, (x_hat.shape[0] if x_hat.dim() == 2 else -1, self.K), "x_hat")
        M = int(x_hat.shape[0])
        if y is None:
            y = _new(stream, (M, self.N), self._f16, x_hat.device)
        elif not (y.is_cuda and y.dtype == self._f16 and y.shape == (M, self.N) and y.is_contiguous()):
            _need(y, self._f16, (M, self.N), "y")
        handle = self._raw_stream(self._dev_index) if stream is None else stream
        self._on = (handle, stream)
        ws = self._workspace(M)
        l1t, wq, ws_, l2, b = self._ptrs
        st = self._fn(x_hat.data_ptr(), l1t, wq, ws_, l2, b, M, self.N, self.K, self.r, self._F, ws.data_ptr(),
                      self._ws_bytes, y.data_ptr(), handle)
        if st != 0:
            raise SvdqError("svdq_linear", st)
        return y
