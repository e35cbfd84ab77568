"""libna: GB300-native multi-dimensional neighborhood attention (NA), forward and backward.

A thin ctypes binding over the C ABI in include/na.h: every function takes torch tensors that
already live on the GPU, checks shapes, and passes raw device pointers, sizes and the current CUDA
stream to the library.  All arithmetic runs in the library's CUDA kernels (tcgen05 tensor-core
kernels for bf16, CUDA-core FMA kernels for fp32); there is no fallback of any kind, and a missing
library raises.

Tensors are contiguous [B, L_1, .., L_n, heads, D] (n = 1..3); lse/delta are fp32 [B, L.., heads].
The unfused operations (na_qk, na_softmax, na_av and their gradients) keep the attention weights
as [B, L.., heads, K], K = the product of the kernel sizes, window offsets first axis outermost.
Around the attention: rotary positions (na_rope), layer norm (na_layernorm), and the window softmax with
dropout or as the difference of two maps (na_softmax_dropout, na_diff_softmax, na_dropout).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

from . import build as _build

__all__ = [
    "NAError", "load", "na_fwd", "na_bwd", "na_bwd_delta", "na_bwd_dq", "na_bwd_dkdv",
    "na_bwd_workspace_size", "na_device_status", "na_strerror", "na_plan_info", "library_path",
    "na_qk", "na_av", "na_softmax", "na_softmax_bwd", "na_qk_bwd", "na_av_bwd", "na_rpb_grad",
    "na_rpb_grad_workspace_size", "na_mask_window", "na_debug_wait_hook",
    "RopeFreqs", "na_rope", "na_rope_bwd", "na_layernorm", "na_layernorm_bwd", "na_layernorm_bwd_workspace_size",
    "na_dropout", "na_softmax_dropout", "na_softmax_dropout_bwd", "na_diff_softmax", "na_diff_softmax_bwd",
    "na_diff_softmax_bwd_workspace_size",
]

NA_BF16, NA_FP32, NA_FP16 = 0, 1, 2
_STATUS = {0: "NA_OK", 1: "NA_ERR_INVALID_ARG", 2: "NA_ERR_UNSUPPORTED", 3: "NA_ERR_ALIGNMENT",
           4: "NA_ERR_CUDA", 5: "NA_ERR_TIMEOUT", 6: "NA_ERR_WORKSPACE"}

_lib = None


class NAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_STATUS.get(status, status)} ({na_strerror(status)})")


def library_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Load libna.so (built by neighborhood_attention_fwd_gb300.build.build()); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"libna.so not found at {path}: run neighborhood_attention_fwd_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    IP = ctypes.POINTER(ctypes.c_int)
    geo = [I, I, IP, I, I]                   # B, ndim, spatial, heads, D
    kd = [IP, IP, F]                         # kernel, dilation, scale
    geo_nd = [I, I, IP, I]                   # B, ndim, spatial, heads
    lib.na_fwd.argtypes = [P, P, P, P, P] + geo + kd + [I, P]
    lib.na_bwd.argtypes = [P, P, P, P, P, P, P, P, P] + geo + kd + [I, P, ctypes.c_size_t, P]
    lib.na_bwd_delta.argtypes = [P, P, P] + geo + [I, P]
    lib.na_bwd_dq.argtypes = [P, P, P, P, P, P, P] + geo + kd + [I, P]
    lib.na_bwd_dkdv.argtypes = [P, P, P, P, P, P, P, P] + geo + kd + [I, P]
    lib.na_bwd_workspace_size.argtypes = [I, I, IP, I]
    lib.na_bwd_workspace_size.restype = ctypes.c_size_t
    lib.na_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
    lib.na_debug_wait_hook.argtypes = [ctypes.c_ulonglong, I]
    lib.na_strerror.argtypes = [I]
    lib.na_strerror.restype = ctypes.c_char_p
    lib.na_plan_info.argtypes = [I, I, I, IP, I, I, IP, IP, ctypes.POINTER(ctypes.c_int64)]
    lib.na_qk.argtypes = [P, P, P, P] + geo + kd + [I, P]
    lib.na_rpb_grad.argtypes = [P, P] + geo_nd + [IP, IP, I, P, ctypes.c_size_t, P]
    lib.na_rpb_grad_workspace_size.argtypes = [I, I, IP, I, IP]
    lib.na_rpb_grad_workspace_size.restype = ctypes.c_size_t
    lib.na_mask_window.argtypes = [P, P] + geo_nd + [IP, IP, I, P]
    lib.na_av.argtypes = [P, P, P] + geo + [IP, IP, I, P]
    lib.na_softmax.argtypes = [P, P] + geo_nd + [IP, I, P]
    lib.na_softmax_bwd.argtypes = [P, P, P] + geo_nd + [IP, I, P]
    lib.na_qk_bwd.argtypes = [P, P, P, P, P] + geo + kd + [I, P]
    lib.na_av_bwd.argtypes = [P, P, P, P, P] + geo + [IP, IP, I, P]
    L, Z, DB = ctypes.c_int64, ctypes.c_size_t, ctypes.c_double
    rope = [P, P, P, P, I, I, IP, I, I, I, IP, ctypes.POINTER(DB), ctypes.POINTER(L), F, I, I, P]
    lib.na_rope.argtypes = lib.na_rope_bwd.argtypes = rope
    lib.na_layernorm.argtypes = [P, P, P, P, P, P, L, I, F, I, P]
    lib.na_layernorm_bwd.argtypes = [P] * 8 + [L, I, I, P, Z, P]
    lib.na_layernorm_bwd_workspace_size.argtypes = [L, I, I]
    lib.na_layernorm_bwd_workspace_size.restype = Z
    drop = [IP, DB, P, I]                    # kernel, p, rng, dtype
    lib.na_dropout.argtypes = [P, P, L, DB, P, I, P]
    lib.na_softmax_dropout.argtypes = [P, P] + geo_nd + drop + [P]
    lib.na_softmax_dropout_bwd.argtypes = [P, P, P] + geo_nd + drop + [P]
    lib.na_diff_softmax.argtypes = [P, P, P, I, P] + geo_nd + drop + [P]
    lib.na_diff_softmax_bwd.argtypes = [P, P, P, I, P, P, P, P] + geo_nd + drop + [P, Z, P]
    lib.na_diff_softmax_bwd_workspace_size.argtypes = [I, I, IP, I, IP]
    lib.na_diff_softmax_bwd_workspace_size.restype = Z
    for f in ("na_rope", "na_rope_bwd", "na_layernorm", "na_layernorm_bwd", "na_dropout", "na_softmax_dropout",
              "na_softmax_dropout_bwd", "na_diff_softmax", "na_diff_softmax_bwd"):
        getattr(lib, f).restype = I
    for f in ("na_fwd", "na_bwd", "na_bwd_delta", "na_bwd_dq", "na_bwd_dkdv", "na_device_status", "na_plan_info",
              "na_qk", "na_av", "na_softmax", "na_softmax_bwd", "na_qk_bwd", "na_av_bwd", "na_rpb_grad",
              "na_mask_window"):
        getattr(lib, f).restype = I
    _lib = lib
    return lib


def na_strerror(status: int) -> str:
    return load().na_strerror(int(status)).decode()


_INT_MAX = 2 ** 31 - 1


def _fits(what, *sizes):
    """Refuses sizes that a C int would cut."""
    if max(sizes, default=0) > _INT_MAX:
        raise NAError(2, f"{what}: a size past 2^31 - 1")


def _ints(vals):
    vals = [int(x) for x in vals]
    _fits("sizes", *vals)
    return (ctypes.c_int * len(vals))(*vals)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return NA_BF16
    if t.dtype == torch.float32:
        return NA_FP32
    if t.dtype == torch.float16:
        return NA_FP16
    raise TypeError(f"unsupported dtype {t.dtype}: use bfloat16, float16 or float32")


def _geometry(q: torch.Tensor):
    if q.dim() < 4 or q.dim() > 6:
        raise ValueError("expected [B, L_1..L_n, heads, D] with n in 1..3")
    _fits("sizes", *q.shape)
    B = q.shape[0]
    spatial = tuple(int(s) for s in q.shape[1:-2])
    return B, len(spatial), spatial, int(q.shape[-2]), int(q.shape[-1])


def _check(t: torch.Tensor, shape, dtype, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ok(status: int, what: str):
    if status != 0:
        raise NAError(status, what)


def _kd(ndim, kernel, dilation):
    kernel = (kernel,) * ndim if isinstance(kernel, int) else tuple(kernel)
    dilation = (1,) * ndim if dilation is None else ((dilation,) * ndim if isinstance(dilation, int) else tuple(dilation))
    if len(kernel) != ndim or len(dilation) != ndim:
        raise ValueError("kernel and dilation need one entry per spatial axis")
    return kernel, dilation


def na_fwd(q, k, v, o, lse, kernel, dilation=None, scale=None, stream=None):
    """O = NA(q, k, v) and the natural-log LSE, written into o and lse."""
    B, ndim, spatial, heads, D = _geometry(q)
    for name, t in (("k", k), ("v", v), ("o", o)):
        _check(t, q.shape, q.dtype, name)
    _check(q, q.shape, q.dtype, "q")
    _check(lse, q.shape[:-1], torch.float32, "lse")
    kernel, dilation = _kd(ndim, kernel, dilation)
    scale = D ** -0.5 if scale is None else float(scale)
    st = load().na_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                       B, ndim, _ints(spatial), heads, D, _ints(kernel), _ints(dilation), scale,
                       _dtype_code(q), _stream(stream))
    _ok(st, "na_fwd")


def na_bwd_workspace_size(B, spatial, heads) -> int:
    return int(load().na_bwd_workspace_size(int(B), len(spatial), _ints(spatial), int(heads)))


def na_bwd(q, k, v, o, dO, lse, dQ, dK, dV, kernel, dilation=None, scale=None, workspace=None, stream=None):
    """dQ, dK, dV of NA for upstream gradient dO (Delta prologue + dQ pass + dK/dV pass)."""
    B, ndim, spatial, heads, D = _geometry(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dO", dO), ("dQ", dQ), ("dK", dK), ("dV", dV)):
        _check(t, q.shape, q.dtype, name)
    _check(lse, q.shape[:-1], torch.float32, "lse")
    kernel, dilation = _kd(ndim, kernel, dilation)
    scale = D ** -0.5 if scale is None else float(scale)
    if workspace is not None:
        _check(workspace, workspace.shape, workspace.dtype, "workspace")
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = load().na_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dO.data_ptr(), lse.data_ptr(),
                       dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), B, ndim, _ints(spatial), heads, D,
                       _ints(kernel), _ints(dilation), scale, _dtype_code(q), ws_ptr, ws_bytes, _stream(stream))
    _ok(st, "na_bwd")


def na_bwd_delta(o, dO, delta, stream=None):
    """delta = <dO, O> per row (fp32)."""
    B, ndim, spatial, heads, D = _geometry(o)
    _check(dO, o.shape, o.dtype, "dO")
    _check(delta, o.shape[:-1], torch.float32, "delta")
    st = load().na_bwd_delta(o.data_ptr(), dO.data_ptr(), delta.data_ptr(), B, ndim, _ints(spatial), heads, D,
                             _dtype_code(o), _stream(stream))
    _ok(st, "na_bwd_delta")


def na_bwd_dq(q, k, v, dO, lse, delta, dQ, kernel, dilation=None, scale=None, stream=None):
    B, ndim, spatial, heads, D = _geometry(q)
    for name, t in (("k", k), ("v", v), ("dO", dO), ("dQ", dQ)):
        _check(t, q.shape, q.dtype, name)
    _check(lse, q.shape[:-1], torch.float32, "lse")
    _check(delta, q.shape[:-1], torch.float32, "delta")
    kernel, dilation = _kd(ndim, kernel, dilation)
    scale = D ** -0.5 if scale is None else float(scale)
    st = load().na_bwd_dq(q.data_ptr(), k.data_ptr(), v.data_ptr(), dO.data_ptr(), lse.data_ptr(), delta.data_ptr(),
                          dQ.data_ptr(), B, ndim, _ints(spatial), heads, D, _ints(kernel), _ints(dilation), scale,
                          _dtype_code(q), _stream(stream))
    _ok(st, "na_bwd_dq")


def na_bwd_dkdv(q, k, v, dO, lse, delta, dK, dV, kernel, dilation=None, scale=None, stream=None):
    B, ndim, spatial, heads, D = _geometry(q)
    for name, t in (("k", k), ("v", v), ("dO", dO), ("dK", dK), ("dV", dV)):
        _check(t, q.shape, q.dtype, name)
    _check(lse, q.shape[:-1], torch.float32, "lse")
    _check(delta, q.shape[:-1], torch.float32, "delta")
    kernel, dilation = _kd(ndim, kernel, dilation)
    scale = D ** -0.5 if scale is None else float(scale)
    st = load().na_bwd_dkdv(q.data_ptr(), k.data_ptr(), v.data_ptr(), dO.data_ptr(), lse.data_ptr(),
                            delta.data_ptr(), dK.data_ptr(), dV.data_ptr(), B, ndim, _ints(spatial), heads, D,
                            _ints(kernel), _ints(dilation), scale, _dtype_code(q), _stream(stream))
    _ok(st, "na_bwd_dkdv")


def na_device_status(stream=None):
    """Synchronise the stream and return (status, raw status word); clears the word."""
    raw = ctypes.c_uint32(0)
    st = load().na_device_status(_stream(stream), ctypes.byref(raw))
    return int(st), int(raw.value)


def na_debug_wait_hook(limit_ns: int = 0, withhold: bool = False) -> None:
    """Test hook: the wait limit of later launches that fetch tiles (the tensor-core kernels, the window softmax with
    dropout and differences, the layer norm's gradients; 0: the 2 s default) and, with withhold, the first CTA's
    first halo chunk or tile left unfilled so that a wait runs out."""
    _ok(load().na_debug_wait_hook(int(limit_ns), 1 if withhold else 0), "na_debug_wait_hook")


PLAN_FIELDS = ("T1", "T2", "T3", "H1", "H2", "H3", "G1", "G2", "G3", "NC", "chunks_max", "ctas", "mma_flops",
               "tmem_cols", "smem_bytes", "chunks_total")


def na_plan_info(which: int, B, spatial, heads, D, kernel, dilation=None) -> dict:
    """Tile plan of the bf16 kernel `which` (0 forward, 1 dQ, 2 dK/dV) for this problem."""
    ndim = len(spatial)
    kernel, dilation = _kd(ndim, kernel, dilation)
    out = (ctypes.c_int64 * 16)()
    st = load().na_plan_info(int(which), int(B), ndim, _ints(spatial), int(heads), int(D), _ints(kernel),
                             _ints(dilation), out)
    _ok(st, "na_plan_info")
    return dict(zip(PLAN_FIELDS, [int(x) for x in out]))


# ---------------------------------------------------------------------------------------------
# Unfused operations: logits, window softmax, weighted sum, and their gradients
# ---------------------------------------------------------------------------------------------

def _window_size(kernel) -> int:
    n = 1
    for x in kernel:
        n *= int(x)
    return n


def _attn_geometry(attn: torch.Tensor, kernel):
    """B, ndim, spatial, heads of an attention-weight tensor [B, L.., heads, K]."""
    if attn.dim() < 4 or attn.dim() > 6:
        raise ValueError("expected attention weights [B, L_1..L_n, heads, K] with n in 1..3")
    ndim = attn.dim() - 3
    kernel = (kernel,) * ndim if isinstance(kernel, int) else tuple(kernel)
    if len(kernel) != ndim:
        raise ValueError("kernel needs one entry per spatial axis")
    if int(attn.shape[-1]) != _window_size(kernel):
        raise ValueError(f"last axis of the attention weights must be {_window_size(kernel)}")
    _fits("sizes", *attn.shape)
    return int(attn.shape[0]), ndim, tuple(int(s) for s in attn.shape[1:-2]), int(attn.shape[-2]), kernel


def _rpb_shape(heads, kernel):
    return (heads,) + tuple(2 * int(x) - 1 for x in kernel)


def na_qk(q, k, attn, kernel, dilation=None, scale=None, stream=None, rpb=None):
    """attn = scale * q . k over each query's window, plus the relative positional bias rpb (fp32
    [heads, 2k_0 - 1, ..]) when given."""
    B, ndim, spatial, heads, D = _geometry(q)
    _check(k, q.shape, q.dtype, "k")
    _check(q, q.shape, q.dtype, "q")
    kernel, dilation = _kd(ndim, kernel, dilation)
    _check(attn, tuple(q.shape[:-1]) + (_window_size(kernel),), q.dtype, "attn")
    if rpb is not None:
        _check(rpb, _rpb_shape(heads, kernel), torch.float32, "rpb")
    scale = D ** -0.5 if scale is None else float(scale)
    st = load().na_qk(q.data_ptr(), k.data_ptr(), None if rpb is None else rpb.data_ptr(), attn.data_ptr(), B,
                      ndim, _ints(spatial), heads, D, _ints(kernel), _ints(dilation), scale, _dtype_code(q),
                      _stream(stream))
    _ok(st, "na_qk")


def na_rpb_grad_workspace_size(B, spatial, heads, kernel) -> int:
    kernel = (kernel,) * len(spatial) if isinstance(kernel, int) else tuple(kernel)
    return int(load().na_rpb_grad_workspace_size(int(B), len(spatial), _ints(spatial), int(heads), _ints(kernel)))


def na_rpb_grad(dattn, drpb, kernel, dilation=None, workspace=None, stream=None):
    """drpb (fp32 [heads, 2k_0 - 1, ..]) = the bias table's gradient given the logits' gradient dattn."""
    B, ndim, spatial, heads, kernel = _attn_geometry(dattn, kernel)
    kernel, dilation = _kd(ndim, kernel, dilation)
    _check(dattn, dattn.shape, dattn.dtype, "dattn")
    _check(drpb, _rpb_shape(heads, kernel), torch.float32, "drpb")
    if workspace is not None:
        _check(workspace, workspace.shape, workspace.dtype, "workspace")
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = load().na_rpb_grad(dattn.data_ptr(), drpb.data_ptr(), B, ndim, _ints(spatial), heads, _ints(kernel),
                            _ints(dilation), _dtype_code(dattn), ws_ptr, ws_bytes, _stream(stream))
    _ok(st, "na_rpb_grad")


def na_av(attn, v, o, kernel, dilation=None, stream=None):
    """o = sum over each query's window of attn * v."""
    B, ndim, spatial, heads, D = _geometry(v)
    _check(v, v.shape, v.dtype, "v")
    _check(o, v.shape, v.dtype, "o")
    kernel, dilation = _kd(ndim, kernel, dilation)
    _check(attn, tuple(v.shape[:-1]) + (_window_size(kernel),), v.dtype, "attn")
    st = load().na_av(attn.data_ptr(), v.data_ptr(), o.data_ptr(), B, ndim, _ints(spatial), heads, D,
                      _ints(kernel), _ints(dilation), _dtype_code(v), _stream(stream))
    _ok(st, "na_av")


def na_softmax(x, y, kernel, stream=None):
    """y = softmax of x over each row's K window weights (y may be x)."""
    B, ndim, spatial, heads, kernel = _attn_geometry(x, kernel)
    _check(x, x.shape, x.dtype, "x")
    _check(y, x.shape, x.dtype, "y")
    st = load().na_softmax(x.data_ptr(), y.data_ptr(), B, ndim, _ints(spatial), heads, _ints(kernel),
                           _dtype_code(x), _stream(stream))
    _ok(st, "na_softmax")


def na_softmax_bwd(y, dy, dx, kernel, stream=None):
    """dx = y * (dy - sum_t y dy), the gradient of the window softmax given its output y."""
    B, ndim, spatial, heads, kernel = _attn_geometry(y, kernel)
    for name, t in (("y", y), ("dy", dy), ("dx", dx)):
        _check(t, y.shape, y.dtype, name)
    st = load().na_softmax_bwd(y.data_ptr(), dy.data_ptr(), dx.data_ptr(), B, ndim, _ints(spatial), heads,
                               _ints(kernel), _dtype_code(y), _stream(stream))
    _ok(st, "na_softmax_bwd")


def na_qk_bwd(dattn, q, k, dq, dk, kernel, dilation=None, scale=None, stream=None):
    """dq, dk of na_qk given the logits' gradient dattn."""
    B, ndim, spatial, heads, D = _geometry(q)
    for name, t in (("q", q), ("k", k), ("dq", dq), ("dk", dk)):
        _check(t, q.shape, q.dtype, name)
    kernel, dilation = _kd(ndim, kernel, dilation)
    _check(dattn, tuple(q.shape[:-1]) + (_window_size(kernel),), q.dtype, "dattn")
    scale = D ** -0.5 if scale is None else float(scale)
    st = load().na_qk_bwd(dattn.data_ptr(), q.data_ptr(), k.data_ptr(), dq.data_ptr(), dk.data_ptr(), B, ndim,
                          _ints(spatial), heads, D, _ints(kernel), _ints(dilation), scale, _dtype_code(q),
                          _stream(stream))
    _ok(st, "na_qk_bwd")


def na_av_bwd(dO, attn, v, dattn, dv, kernel, dilation=None, stream=None):
    """dattn, dv of na_av given the output's gradient dO."""
    B, ndim, spatial, heads, D = _geometry(v)
    for name, t in (("dO", dO), ("v", v), ("dv", dv)):
        _check(t, v.shape, v.dtype, name)
    kernel, dilation = _kd(ndim, kernel, dilation)
    K = _window_size(kernel)
    _check(attn, tuple(v.shape[:-1]) + (K,), v.dtype, "attn")
    _check(dattn, tuple(v.shape[:-1]) + (K,), v.dtype, "dattn")
    st = load().na_av_bwd(dO.data_ptr(), attn.data_ptr(), v.data_ptr(), dattn.data_ptr(), dv.data_ptr(), B, ndim,
                          _ints(spatial), heads, D, _ints(kernel), _ints(dilation), _dtype_code(v),
                          _stream(stream))
    _ok(st, "na_av_bwd")


def na_mask_window(attn, sizes, kernel, dilation=None, stream=None):
    """Set, in place, the logits outside each query's variable window to -inf.  sizes: one sequence or
    tensor per axis, sizes[a][x] = the kernel size (odd, <= kernel[a]) of the queries at position x."""
    B, ndim, spatial, heads, kernel = _attn_geometry(attn, kernel)
    kernel, dilation = _kd(ndim, kernel, dilation)
    _check(attn, attn.shape, attn.dtype, "attn")
    if len(sizes) != ndim:
        raise ValueError("sizes needs one entry per spatial axis")
    parts = [torch.as_tensor(sz, dtype=torch.int32, device="cpu").reshape(-1) for sz in sizes]
    for L, part in zip(spatial, parts):
        if part.numel() != L:
            raise ValueError("sizes[a] needs one entry per position along axis a")
    # a copy from pageable host memory has finished when .to() returns, so the sizes are in place
    # whichever stream the kernel runs on; the temporary must then outlive the launch on that stream
    flat = torch.cat(parts).contiguous().to(attn.device)
    st = load().na_mask_window(attn.data_ptr(), flat.data_ptr(), B, ndim, _ints(spatial), heads, _ints(kernel),
                               _ints(dilation), _dtype_code(attn), _stream(stream))
    _ok(st, "na_mask_window")
    if isinstance(stream, torch.cuda.Stream):
        flat.record_stream(stream)
    elif stream is not None:
        torch.cuda.ExternalStream(int(stream)).synchronize()


# ---------------------------------------------------------------------------------------------
# Around the attention: rotary positions, layer norm, dropout, differential weights
# ---------------------------------------------------------------------------------------------

# These operators are small beside the attention, so their calls are kept short: sizes become C arrays once per
# size, and the checks and the stream take the shortest way through torch.

@functools.lru_cache(maxsize=1024)
def _sizes(vals):
    """A C int array of a tuple of sizes."""
    _fits("sizes", *vals)
    return (ctypes.c_int * len(vals))(*vals)


@functools.lru_cache(maxsize=1024)
def _grid(shape):
    """The spatial axes of [B, L.., heads, D] as a C int array."""
    _fits("sizes", *shape)
    return _sizes(shape[1:-2])


@functools.lru_cache(maxsize=1024)
def _origins(vals):
    """A C int64 array of a grid's first positions."""
    if not all(-2 ** 63 <= v < 2 ** 63 for v in vals):
        raise ValueError("origin must fit 64 bits")
    return (ctypes.c_int64 * len(vals))(*vals)


def _like(t, shape, dtype, name):
    """A contiguous tensor of this shape and type."""
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        _check(t, shape, dtype, name)


def _launch_stream(stream, *tensors):
    """The raw stream of a call, every tensor being on the current CUDA device (kernels are launched there)."""
    here = -1
    for t in tensors:
        if t is None:
            continue
        at = t.get_device()
        if at < 0:
            raise ValueError("expected CUDA tensors")
        if here < 0:
            here = torch._C._cuda_getDevice()
        if at != here:
            raise ValueError(f"tensor on {t.device}, but the current device is cuda:{here}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(here)
    return _stream(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _workspace(ws, stream, need, device):
    """(tensor, pointer, bytes) of a call's workspace.  Without one from the caller, a call on the current stream
    takes it from torch's allocator, which keeps freed memory at hand; a call on another stream leaves it to the
    library, which allocates on that stream."""
    if ws is None and stream is None:
        n = need()
        if n == 0:
            return None, None, 0
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        return ws, ws.data_ptr(), n
    if ws is None:
        return None, None, 0
    if not ws.is_contiguous():   # a broadcast view has fewer bytes than its elements
        raise ValueError("workspace must be contiguous")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


_CODES = {torch.bfloat16: NA_BF16, torch.float32: NA_FP32, torch.float16: NA_FP16}


def _code(t):
    code = _CODES.get(t.dtype)
    return _dtype_code(t) if code is None else code


class RopeFreqs:
    """Frequencies of na_rope: freqs[a][i] = radians per position of pair i of axis a (axis a owns
    2 len(freqs[a]) channels), the amplitude that scales the rotated channels, and the pairs' layout, "half" or
    "interleaved".  A program makes one per configuration and keeps it."""

    def __init__(self, freqs, amplitude: float = 1.0, layout: str = "half"):
        if layout not in ("half", "interleaved"):
            raise ValueError("layout must be 'half' or 'interleaved'")
        self.freqs = tuple(tuple(float(f) for f in axis) for axis in freqs)
        self.amplitude = float(amplitude)
        self.layout = layout
        flat = [f for axis in self.freqs for f in axis]
        self._rot = (ctypes.c_int * len(self.freqs))(*[2 * len(axis) for axis in self.freqs])
        self._freq = (ctypes.c_double * max(1, len(flat)))(*flat)
        self._code = 0 if layout == "half" else 1

    @classmethod
    def scaled(cls, rot, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, trained: int | None = None,
               fast: float = 32.0, slow: float = 1.0, amplitude: float | None = None, layout: str = "half"):
        """The usual frequencies base^(-2i/r) of rot[a] = r channels per axis, and their scalings for grids or
        sequences `factor` times as long as the trained ones:
          "linear": every frequency divided by factor (positions interpolated);
          "ntk":    base * factor^(r/(r-2)), which divides the lowest frequency by factor and keeps the highest;
          "yarn":   divided by factor where a pair makes at most `slow` turns over the `trained` positions, kept
                    where it makes at least `fast`, blended linearly in the turns between, and the amplitude
                    0.1 ln(factor) + 1 unless one is given."""
        if scaling not in ("none", "linear", "ntk", "yarn"):
            raise ValueError("scaling must be 'none', 'linear', 'ntk' or 'yarn'")
        if not (base > 0 and factor > 0):
            raise ValueError("base and factor must be positive")
        if scaling == "yarn" and (trained is None or trained < 1 or not fast > slow):
            raise ValueError("yarn needs the trained length, and fast > slow")
        axes = []
        for r in rot:
            r = int(r)
            if r < 0 or r % 2:
                raise ValueError("rot must be even")
            b = base * factor ** (r / (r - 2)) if scaling == "ntk" and r > 2 else base
            f = [b ** (-2.0 * i / r) for i in range(r // 2)]
            if scaling == "linear":
                f = [x / factor for x in f]
            elif scaling == "yarn":
                keep = [min(1.0, max(0.0, (trained * x / (2 * math.pi) - slow) / (fast - slow))) for x in f]
                f = [x / factor * (1 - g) + x * g for x, g in zip(f, keep)]
            axes.append(f)
        if amplitude is None:
            amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
        return cls(axes, amplitude, layout)


def _rope(call, what, q, k, q_out, k_out, freqs, origin, stream):
    shape = q.shape
    ndim = len(shape) - 3
    if ndim < 1 or ndim > 3:
        raise ValueError("expected [B, L_1..L_n, heads, D] with n in 1..3")
    if len(freqs._rot) != ndim:
        raise ValueError("the frequencies need one entry per spatial axis")
    dtype = q.dtype
    _like(q, shape, dtype, "q")
    _like(q_out, shape, dtype, "q_out")
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    heads_k = 0
    if k is not None:
        shape_k = k.shape
        if shape_k != shape and (len(shape_k) != ndim + 3 or shape_k[:-2] != shape[:-2] or shape_k[-1] != shape[-1]):
            raise ValueError("k must have the axes of q but for the heads")
        heads_k = shape_k[-2]
        if heads_k > _INT_MAX:
            _fits(what, heads_k)
        _like(k, shape_k, dtype, "k")
        _like(k_out, shape_k, dtype, "k_out")
    stream = _launch_stream(stream, q, k, q_out, k_out)
    if origin is not None:
        origin = _origins((origin,) * ndim if isinstance(origin, int) else tuple(map(int, origin)))
        if len(origin) != ndim:
            raise ValueError("origin needs one entry per spatial axis")
    st = call(q.data_ptr(), _ptr(k), q_out.data_ptr(), _ptr(k_out), shape[0], ndim, _grid(shape), shape[-2],
              heads_k, shape[-1], freqs._rot, freqs._freq, origin, freqs.amplitude, freqs._code, _code(q), stream)
    if st:
        _ok(st, what)


def na_rope(q, k, q_out, k_out, freqs: RopeFreqs, origin=None, stream=None):
    """Rotary positions of q [B, L.., heads, D] and k (the same with its own head count, or None), written
    into q_out and k_out, which may be q and k.  origin: the grid's first position, one per axis or one for all."""
    _rope(load().na_rope, "na_rope", q, k, q_out, k_out, freqs, origin, stream)


def na_rope_bwd(dq_out, dk_out, dq, dk, freqs: RopeFreqs, origin=None, stream=None):
    """dq, dk of na_rope given its outputs' gradients (dq may be dq_out, dk may be dk_out)."""
    _rope(load().na_rope_bwd, "na_rope_bwd", dq_out, dk_out, dq, dk, freqs, origin, stream)


def _rows(x):
    shape = x.shape
    n = x.numel()
    if not shape or n == 0:
        raise ValueError("expected [.., C] with at least one element")
    if shape[-1] > _INT_MAX:
        _fits("channels", shape[-1])
    return shape, n // shape[-1], shape[-1]


def _vectors(C, **named):
    """fp32 [C] tensors, or None."""
    for name, t in named.items():
        if t is not None:
            _like(t, (C,), torch.float32, name)


def _statistics(shape, mean, rstd):
    lead = shape[:-1]
    _like(mean, lead, torch.float32, "mean")
    _like(rstd, lead, torch.float32, "rstd")


def na_layernorm(x, w, b, y, mean=None, rstd=None, eps: float = 1e-5, stream=None):
    """y = (x - mean) * rstd * w + b over the last axis of x [.., C] (per head: [B, L.., heads, D]; per token:
    [B, L.., heads * D]).  w, b: fp32 [C] or None; mean, rstd: fp32 x.shape[:-1] for the backward, or None."""
    shape, rows, C = _rows(x)
    _like(x, shape, x.dtype, "x")
    _like(y, shape, x.dtype, "y")
    _vectors(C, w=w, b=b)
    if (mean is None) != (rstd is None):
        raise ValueError("mean and rstd go together")
    if mean is not None:
        _statistics(shape, mean, rstd)
    stream = _launch_stream(stream, x, w, b, y, mean, rstd)
    st = load().na_layernorm(x.data_ptr(), _ptr(w), _ptr(b), y.data_ptr(), _ptr(mean), _ptr(rstd), rows, C, eps, _code(x),
                             stream)
    _ok(st, "na_layernorm")


@functools.lru_cache(maxsize=1024)
def _norm_need(rows, C, code):
    return int(load().na_layernorm_bwd_workspace_size(rows, C, code))


def na_layernorm_bwd_workspace_size(rows: int, C: int, dtype=torch.bfloat16) -> int:
    return _norm_need(int(rows), int(C), _CODES[dtype]) if int(C) <= _INT_MAX else 0


def na_layernorm_bwd(dy, x, w, mean, rstd, dx, dw=None, db=None, workspace=None, stream=None):
    """dx (may be dy or x) and, when given, dw and db (fp32 [C]) of na_layernorm."""
    shape, rows, C = _rows(x)
    dtype = x.dtype
    _like(x, shape, dtype, "x")
    _like(dy, shape, dtype, "dy")
    _like(dx, shape, dtype, "dx")
    _vectors(C, w=w, dw=dw, db=db)
    if (dw is None) != (db is None):
        raise ValueError("dw and db go together")
    _statistics(shape, mean, rstd)
    raw = _launch_stream(stream, dy, x, w, mean, rstd, dx, dw, db, workspace)
    code = _code(x)
    ws, ws_ptr, ws_bytes = (None, None, 0) if dw is None else _workspace(
        workspace, stream, lambda: _norm_need(rows, C, code), x.device)
    st = load().na_layernorm_bwd(dy.data_ptr(), x.data_ptr(), _ptr(w), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(),
                                 _ptr(dw), _ptr(db), rows, C, code, ws_ptr, ws_bytes, raw)
    _ok(st, "na_layernorm_bwd")


def _rng(rng):
    if rng is not None:
        _like(rng, (2,), torch.int64, "rng")
    return _ptr(rng)


@functools.lru_cache(maxsize=1024)
def _window_of(shape, kernel):
    """B, ndim, the grid and the kernel as C arrays, and the heads between them, of weights [B, L.., heads, K]."""
    ndim = len(shape) - 3
    if ndim < 1 or ndim > 3:
        raise ValueError("expected attention weights [B, L_1..L_n, heads, K] with n in 1..3")
    kernel = (kernel,) * ndim if isinstance(kernel, int) else kernel
    if len(kernel) != ndim:
        raise ValueError("kernel needs one entry per spatial axis")
    if shape[-1] != math.prod(kernel):
        raise ValueError(f"last axis of the attention weights must be {math.prod(kernel)}")
    _fits("sizes", *shape)
    return shape[0], ndim, _sizes(tuple(shape[1:-2])), shape[-2], _sizes(kernel)


def _window(x, kernel):
    return _window_of(x.shape, kernel if isinstance(kernel, int) else tuple(map(int, kernel)))


def na_dropout(x, y, p: float, rng, stream=None):
    """y = dropout(x) (y may be x): each element zero with probability p, else scaled.  rng: int64 CUDA tensor
    (seed, offset); the same state keeps the same elements, so the gradient is na_dropout(dy, dx, p, rng)."""
    _like(x, x.shape, x.dtype, "x")
    _like(y, x.shape, x.dtype, "y")
    state = _rng(rng)
    stream = _launch_stream(stream, x, y, rng)
    st = load().na_dropout(x.data_ptr(), y.data_ptr(), x.numel(), p, state, _code(x), stream)
    _ok(st, "na_dropout")


def na_softmax_dropout(x, y, kernel, p: float, rng, stream=None):
    """y = dropout(softmax(x)) over each row's K window weights (y may be x; keep x for the gradient)."""
    B, ndim, grid, heads, kern = _window(x, kernel)
    _like(x, x.shape, x.dtype, "x")
    _like(y, x.shape, x.dtype, "y")
    state = _rng(rng)
    stream = _launch_stream(stream, x, y, rng)
    st = load().na_softmax_dropout(x.data_ptr(), y.data_ptr(), B, ndim, grid, heads, kern, p, state, _code(x), stream)
    _ok(st, "na_softmax_dropout")


def na_softmax_dropout_bwd(x, dy, dx, kernel, p: float, rng, stream=None):
    """dx of na_softmax_dropout given its logits x, dy and the forward's p and rng (dx may be x or dy)."""
    B, ndim, grid, heads, kern = _window(x, kernel)
    for name, t in (("x", x), ("dy", dy), ("dx", dx)):
        _like(t, x.shape, x.dtype, name)
    state = _rng(rng)
    stream = _launch_stream(stream, x, dy, dx, rng)
    st = load().na_softmax_dropout_bwd(x.data_ptr(), dy.data_ptr(), dx.data_ptr(), B, ndim, grid, heads, kern, p, state,
                                       _code(x), stream)
    _ok(st, "na_softmax_dropout_bwd")


def _lam_rows(lam, rows_shape, heads):
    """0 for a weight per head ([heads]), 1 for one per row ([B, L.., heads])."""
    per_row = lam.dim() != 1
    _like(lam, rows_shape if per_row else (heads,), torch.float32, "lam")
    return int(per_row)


def na_diff_softmax(x1, x2, lam, y, kernel, p: float = 0.0, rng=None, stream=None):
    """y = dropout(softmax(x1) - lam * softmax(x2)) over each row's K window weights.  lam: fp32 [heads] or
    [B, L.., heads].  y may be x1 or x2 (keep the logits for the gradient)."""
    B, ndim, grid, heads, kern = _window(x1, kernel)
    for name, t in (("x1", x1), ("x2", x2), ("y", y)):
        _like(t, x1.shape, x1.dtype, name)
    per_row = _lam_rows(lam, x1.shape[:-1], heads)
    state = _rng(rng)
    stream = _launch_stream(stream, x1, x2, lam, y, rng)
    st = load().na_diff_softmax(x1.data_ptr(), x2.data_ptr(), lam.data_ptr(), per_row, y.data_ptr(), B, ndim, grid, heads, kern,
                                p, state, _code(x1), stream)
    _ok(st, "na_diff_softmax")


def na_diff_softmax_bwd_workspace_size(B, spatial, heads, kernel) -> int:
    kernel = (kernel,) * len(spatial) if isinstance(kernel, int) else tuple(kernel)
    if max(int(B), int(heads), *map(int, spatial), *map(int, kernel)) > _INT_MAX:
        return 0
    return int(load().na_diff_softmax_bwd_workspace_size(int(B), len(spatial), _ints(spatial), int(heads), _ints(kernel)))


def na_diff_softmax_bwd(x1, x2, lam, dy, dx1, dx2, dlam, kernel, p: float = 0.0, rng=None, workspace=None, stream=None):
    """dx1, dx2, dlam (the shape of lam) of na_diff_softmax given its logits, dy and the forward's p and rng."""
    B, ndim, grid, heads, kern = _window(x1, kernel)
    for name, t in (("x1", x1), ("x2", x2), ("dy", dy), ("dx1", dx1), ("dx2", dx2)):
        _like(t, x1.shape, x1.dtype, name)
    per_row = _lam_rows(lam, x1.shape[:-1], heads)
    _like(dlam, lam.shape, torch.float32, "dlam")
    state = _rng(rng)
    raw = _launch_stream(stream, x1, x2, lam, dy, dx1, dx2, dlam, rng, workspace)
    ws, ws_ptr, ws_bytes = (None, None, 0) if per_row else _workspace(
        workspace, stream, lambda: load().na_diff_softmax_bwd_workspace_size(B, ndim, grid, heads, kern), x1.device)
    st = load().na_diff_softmax_bwd(x1.data_ptr(), x2.data_ptr(), lam.data_ptr(), per_row, dy.data_ptr(), dx1.data_ptr(),
                                    dx2.data_ptr(), dlam.data_ptr(), B, ndim, grid, heads, kern, p, state, _code(x1),
                                    ws_ptr, ws_bytes, raw)
    _ok(st, "na_diff_softmax_bwd")
