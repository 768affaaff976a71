"""ctypes binding of libtg.so: the same entry points as include/tg.h.

Each function takes torch CUDA tensors, checks that their shapes agree,
allocates the output (and the workspace the call asks for) with torch's
caching allocator when the caller passes none, and calls the C entry point on
the current CUDA stream.  No arithmetic happens here: every product runs in
the library's kernels.  If libtg.so has not been built the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtg.so")
DEFAULT_TABLE = os.path.join(_PKG, "tables", "gb300.txt")
_lock = threading.Lock()
_lib = None

TG_BF16, TG_F16, TG_F32 = 0, 1, 2
_DT = {torch.bfloat16: TG_BF16, torch.float16: TG_F16, torch.float32: TG_F32}

TG_OP_GEMM_FWD, TG_OP_GEMM_DGRAD, TG_OP_GEMM_WGRAD = 0, 1, 2
TG_OP_LORA_DOWN, TG_OP_LORA_UP, TG_OP_LORA_GRAD, TG_OP_BMM_ATTN = 3, 4, 5, 6
TG_OP_LORA_DOWN_F32W, TG_OP_LORA_UP_F32W, TG_OP_LORA_GRAD_F32W = 7, 8, 9
TG_OP_ATTN_BWD = 10
TG_OP_GEMM_FWD_LORA, TG_OP_GEMM_DGRAD_LORA = 11, 12
TG_OP_GROUPED_FWD, TG_OP_GROUPED_DGRAD, TG_OP_GROUPED_WGRAD, TG_OP_GROUPED_UNALIGNED = 13, 14, 15, 16
TG_OP_NORM_RESIDUAL_BWD, TG_OP_GRAD_CLIP = 17, 18
TG_OP_LAYER_NORM_BWD, TG_OP_GATED_FWD, TG_OP_GATED_BWD, TG_OP_GATED_UNALIGNED, TG_OP_ORTHOGONALIZE = 19, 20, 21, 22, 23
TG_GATE_NONE, TG_GATE_CHANNEL, TG_GATE_TOKEN, TG_GATE_FULL = 0, 1, 2, 3
ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
ATTN_OPS = {"qk": 0, "pv": 1, "do_vt": 2, "pt_do": 3, "ds_k": 4, "dst_q": 5}
SIZE_MAX = (1 << 64) - 1

# every symbol include/tg.h declares, with (restype, argtypes)
_vp, _i64, _sz, _i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
SIGNATURES = {
    "tg_gemm_fwd": (_i, [_vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_gemm_dgrad": (_i, [_vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_gemm_wgrad": (_i, [_vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_gemm_fwd_lora": (_i, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, ctypes.c_float, _i, _i, _vp, _sz, _vp]),
    "tg_gemm_dgrad_lora": (_i, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, ctypes.c_float, _i, _i, _vp, _sz,
                                _vp]),
    "tg_gemm_wgrad_accumulate": (_i, [_vp, _vp, _vp, _i64, _i64, _i64, _i, _vp, _sz, _vp]),
    "tg_gemm_wgrad_noalloc": (_i, [_vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _vp]),
    "tg_lora_down": (_i, [_vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_lora_up": (_i, [_vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_lora_up_add": (_i, [_vp, _vp, _vp, _i64, _i64, _i64, ctypes.c_float, _i, _i, _vp, _sz, _vp]),
    "tg_lora_grad": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i, _i,
                          _vp, _sz, _vp]),
    "tg_lora_down_f32w": (_i, [_vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_lora_up_f32w": (_i, [_vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_lora_grad_f32w": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i, _i,
                               _vp, _sz, _vp]),
    "tg_attn_fwd": (_i, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, ctypes.c_float, _i, _i, _vp]),
    "tg_attn_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, ctypes.c_float, _i, _i, _vp, _sz, _vp]),
    "tg_lora_grad_add": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, ctypes.c_float,
                              _i, _i, _vp, _sz, _vp]),
    "tg_bmm_attn": (_i, [_i, _vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_grouped_fwd": (_i, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_grouped_dgrad": (_i, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_grouped_wgrad": (_i, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_norm_residual_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _i64, _i64, ctypes.c_float,
                                  ctypes.c_float, _i, _i, _vp]),
    "tg_norm_residual_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                  ctypes.c_float, _i, _i, _i, _vp, _sz, _vp]),
    "tg_grad_norm": (_i, [_vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp]),
    "tg_grad_clip": (_i, [_vp, _vp, _vp, _vp, _i64, ctypes.c_float, _vp, _vp, _sz, _vp]),
    "tg_layer_norm_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, ctypes.c_float, _i, _vp]),
    "tg_layer_norm_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_gated_fwd": (_i, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_gated_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i, _i, _vp, _sz, _vp]),
    "tg_orthogonalize": (_i, [_vp, _vp, _i64, _i64, _i64, _vp, _i64, ctypes.c_float, ctypes.c_float, _i, _i, _vp, _sz,
                              _vp]),
    "tg_workspace_size": (_sz, [_i, _i64, _i64, _i64, _i64, _i, _i]),
    "tg_stream_status": (_i, [_vp]),
    "tg_status_string": (ctypes.c_char_p, [_i]),
    "tg_load_table": (_i, [ctypes.c_char_p]),
    "tg_version": (_i, []),
    "tg_last_call": (_sz, [ctypes.c_char_p, _sz]),
    "tg_plan_describe": (_sz, [_i, _i64, _i64, _i64, _i64, _i, _i, _i, ctypes.c_char_p, _sz]),
    "tg_wait_probe": (_i, [_i64, _vp]),
}


class TGError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = status
        super().__init__(f"{where}: tg status {status} ({lib().tg_status_string(status).decode()})")


def lib() -> ctypes.CDLL:
    """The loaded libtg.so (built in-tree by gemms_linear_layers_gb300.build)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m gemms_linear_layers_gb300.build` (needs nvcc)")
            l = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(l, name)
                fn.restype = res
                fn.argtypes = args
            _lib = l
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise TGError(status, where)


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _keep(buf, stream):
    """A workspace allocated here is freed on return; tell the caching
    allocator which stream still uses it."""
    if buf is not None and stream is not None:
        buf.record_stream(stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None and t.numel() > 0 else ctypes.c_void_p(0)


def _need(t, name, ndim):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor, got shape {tuple(t.shape)}")
    return t


def _out(out, shape, dtype, device, name):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(out, name, len(shape))
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype}, got {tuple(out.shape)} {out.dtype}")
    return out


def _workspace(op, dims, din, dout, ws, device):
    n = lib().tg_workspace_size(op, *dims, din, dout)
    if n == SIZE_MAX:
        raise ValueError(f"invalid sizes {dims} for workspace query {op}")
    if n == 0:
        return ctypes.c_void_p(0), 0, None
    if ws is not None and ws.numel() * ws.element_size() >= n:
        return ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size(), ws
    buf = torch.empty(n, dtype=torch.uint8, device=device)
    return ctypes.c_void_p(buf.data_ptr()), n, buf


# --------------------------------------------------------------------------
def tg_gemm_fwd(X, W, Y=None, out_dtype=None, ws=None, stream=None):
    """Y[T, d_out] = X[T, d_in] W[d_out, d_in]^T."""
    _need(X, "X", 2), _need(W, "W", 2)
    T, d_in = X.shape
    d_out = W.shape[0]
    if W.shape[1] != d_in or W.dtype != X.dtype:
        raise ValueError("W must be [d_out, d_in] with X's dtype")
    Y = _out(Y, (T, d_out), out_dtype or X.dtype, X.device, "Y")
    wp, wn, keep = _workspace(TG_OP_GEMM_FWD, (T, d_out, d_in, 0), _DT[X.dtype], _DT[Y.dtype], ws, X.device)
    _check(lib().tg_gemm_fwd(_ptr(X), _ptr(W), _ptr(Y), T, d_out, d_in, _DT[X.dtype], _DT[Y.dtype], wp, wn,
                             _stream(stream)), "tg_gemm_fwd")
    _keep(keep, stream)
    return Y


def tg_gemm_dgrad(dY, W, dX=None, out_dtype=None, ws=None, stream=None):
    """dX[T, d_in] = dY[T, d_out] W[d_out, d_in]."""
    _need(dY, "dY", 2), _need(W, "W", 2)
    T, d_out = dY.shape
    d_in = W.shape[1]
    if W.shape[0] != d_out or W.dtype != dY.dtype:
        raise ValueError("W must be [d_out, d_in] with dY's dtype")
    dX = _out(dX, (T, d_in), out_dtype or dY.dtype, dY.device, "dX")
    wp, wn, keep = _workspace(TG_OP_GEMM_DGRAD, (T, d_out, d_in, 0), _DT[dY.dtype], _DT[dX.dtype], ws, dY.device)
    _check(lib().tg_gemm_dgrad(_ptr(dY), _ptr(W), _ptr(dX), T, d_out, d_in, _DT[dY.dtype], _DT[dX.dtype], wp, wn,
                               _stream(stream)), "tg_gemm_dgrad")
    _keep(keep, stream)
    return dX


def tg_gemm_wgrad(dY, X, dW=None, out_dtype=None, ws=None, stream=None):
    """dW[d_out, d_in] = dY[T, d_out]^T X[T, d_in]."""
    _need(dY, "dY", 2), _need(X, "X", 2)
    T, d_out = dY.shape
    d_in = X.shape[1]
    if X.shape[0] != T or X.dtype != dY.dtype:
        raise ValueError("X must be [T, d_in] with dY's dtype")
    dW = _out(dW, (d_out, d_in), out_dtype or dY.dtype, dY.device, "dW")
    wp, wn, keep = _workspace(TG_OP_GEMM_WGRAD, (T, d_out, d_in, 0), _DT[dY.dtype], _DT[dW.dtype], ws, dY.device)
    _check(lib().tg_gemm_wgrad(_ptr(dY), _ptr(X), _ptr(dW), T, d_out, d_in, _DT[dY.dtype], _DT[dW.dtype], wp, wn,
                               _stream(stream)), "tg_gemm_wgrad")
    _keep(keep, stream)
    return dW



def tg_gemm_fwd_lora(X, W, H, B, scale, Y=None, out_dtype=None, ws=None, stream=None):
    """Y = X W^T + scale H B^T in one product: X [T, d_in], W [d_out, d_in], H [T, r], B [d_out, r]."""
    _need(X, "X", 2)
    _need(W, "W", 2)
    _need(H, "H", 2)
    _need(B, "B", 2)
    T, d_in = X.shape
    d_out, r = W.shape[0], H.shape[1]
    if W.shape[1] != d_in or H.shape[0] != T or tuple(B.shape) != (d_out, r):
        raise ValueError("shapes do not match")
    if not (W.dtype == H.dtype == B.dtype == X.dtype):
        raise ValueError("X, W, H, B must share a dtype")
    Y = _out(Y, (T, d_out), out_dtype or X.dtype, X.device, "Y")
    wp, wn, keep = _workspace(TG_OP_GEMM_FWD_LORA, (T, d_out, d_in, r), _DT[X.dtype], _DT[Y.dtype], ws, X.device)
    _check(lib().tg_gemm_fwd_lora(_ptr(X), _ptr(W), _ptr(H), _ptr(B), _ptr(Y), T, d_out, d_in, r, float(scale),
                                  _DT[X.dtype], _DT[Y.dtype], wp, wn, _stream(stream)), "tg_gemm_fwd_lora")
    _keep(keep, stream)
    return Y


def tg_gemm_dgrad_lora(dY, W, dH, A, scale, dX=None, out_dtype=None, ws=None, stream=None):
    """dX = dY W + scale dH A in one product: dY [T, d_out], W [d_out, d_in], dH [T, r] FP32, A [r, d_in]."""
    _need(dY, "dY", 2)
    _need(W, "W", 2)
    _need(A, "A", 2)
    T, d_out = dY.shape
    d_in, r = W.shape[1], A.shape[0]
    if W.shape[0] != d_out or A.shape[1] != d_in or tuple(dH.shape) != (T, r):
        raise ValueError("shapes do not match")
    if dH.dtype != torch.float32 or not dH.is_contiguous() or dH.device != dY.device:
        raise ValueError("dH must be a contiguous FP32 tensor on the device of dY")
    if not (W.dtype == A.dtype == dY.dtype):
        raise ValueError("dY, W, A must share a dtype")
    dX = _out(dX, (T, d_in), out_dtype or dY.dtype, dY.device, "dX")
    wp, wn, keep = _workspace(TG_OP_GEMM_DGRAD_LORA, (T, d_out, d_in, r), _DT[dY.dtype], _DT[dX.dtype], ws, dY.device)
    _check(lib().tg_gemm_dgrad_lora(_ptr(dY), _ptr(W), _ptr(dH), _ptr(A), _ptr(dX), T, d_out, d_in, r, float(scale),
                                    _DT[dY.dtype], _DT[dX.dtype], wp, wn, _stream(stream)), "tg_gemm_dgrad_lora")
    _keep(keep, stream)
    return dX


def tg_gemm_wgrad_accumulate(dY, X, dW, ws=None, stream=None):
    """dW[d_out, d_in] += dY[T, d_out]^T X[T, d_in], dW an FP32 tensor."""
    _need(dY, "dY", 2), _need(X, "X", 2)
    T, d_out = dY.shape
    d_in = X.shape[1]
    if X.shape[0] != T or X.dtype != dY.dtype:
        raise ValueError("X must be [T, d_in] with dY's dtype")
    if dW is None or dW.dtype != torch.float32 or tuple(dW.shape) != (d_out, d_in) or not dW.is_contiguous():
        raise ValueError("dW must be a contiguous FP32 [d_out, d_in] tensor")
    wp, wn, keep = _workspace(TG_OP_GEMM_WGRAD, (T, d_out, d_in, 0), _DT[dY.dtype], _DT[torch.float32], ws, dY.device)
    _check(lib().tg_gemm_wgrad_accumulate(_ptr(dY), _ptr(X), _ptr(dW), T, d_out, d_in, _DT[dY.dtype], wp, wn,
                                          _stream(stream)), "tg_gemm_wgrad_accumulate")
    _keep(keep, stream)
    return dW
def tg_gemm_wgrad_noalloc(dY, X, dW, stream=None):
    """dW = dY^T X without any device allocation by the library (the split-K
    scratch is the library's own static array); dW must be given."""
    _need(dY, "dY", 2), _need(X, "X", 2), _need(dW, "dW", 2)
    T, d_out = dY.shape
    d_in = X.shape[1]
    if X.shape[0] != T or X.dtype != dY.dtype or tuple(dW.shape) != (d_out, d_in):
        raise ValueError("inconsistent shapes or dtypes")
    _check(lib().tg_gemm_wgrad_noalloc(_ptr(dY), _ptr(X), _ptr(dW), T, d_out, d_in, _DT[dY.dtype], _DT[dW.dtype],
                                       _stream(stream)), "tg_gemm_wgrad_noalloc")
    return dW


def tg_lora_down(X, A, H=None, out_dtype=None, ws=None, stream=None):
    """H[T, r] = X[T, d_in] A[r, d_in]^T."""
    _need(X, "X", 2), _need(A, "A", 2)
    T, d_in = X.shape
    r = A.shape[0]
    if A.shape[1] != d_in or A.dtype != X.dtype:
        raise ValueError("A must be [r, d_in] with X's dtype")
    H = _out(H, (T, r), out_dtype or X.dtype, X.device, "H")
    wp, wn, keep = _workspace(TG_OP_LORA_DOWN, (T, d_in, r, 0), _DT[X.dtype], _DT[H.dtype], ws, X.device)
    _check(lib().tg_lora_down(_ptr(X), _ptr(A), _ptr(H), T, d_in, r, _DT[X.dtype], _DT[H.dtype], wp, wn,
                              _stream(stream)), "tg_lora_down")
    _keep(keep, stream)
    return H


def tg_lora_up(H, B, Y=None, out_dtype=None, ws=None, stream=None):
    """Y[T, d_out] = H[T, r] B[d_out, r]^T."""
    _need(H, "H", 2), _need(B, "B", 2)
    T, r = H.shape
    d_out = B.shape[0]
    if B.shape[1] != r or B.dtype != H.dtype:
        raise ValueError("B must be [d_out, r] with H's dtype")
    Y = _out(Y, (T, d_out), out_dtype or H.dtype, H.device, "Y")
    wp, wn, keep = _workspace(TG_OP_LORA_UP, (T, d_out, r, 0), _DT[H.dtype], _DT[Y.dtype], ws, H.device)
    _check(lib().tg_lora_up(_ptr(H), _ptr(B), _ptr(Y), T, d_out, r, _DT[H.dtype], _DT[Y.dtype], wp, wn,
                            _stream(stream)), "tg_lora_up")
    _keep(keep, stream)
    return Y



def tg_lora_up_add(H, B, Y, scale, ws=None, stream=None):
    """Y[T, d_out] += scale * H[T, r] B[d_out, r]^T (one rounding to Y's type)."""
    _need(H, "H", 2), _need(B, "B", 2)
    T, r = H.shape
    d_out = B.shape[0]
    if B.shape[1] != r or B.dtype != H.dtype:
        raise ValueError("B must be [d_out, r] with H's dtype")
    if Y is None or tuple(Y.shape) != (T, d_out) or not Y.is_contiguous():
        raise ValueError("Y must be a contiguous [T, d_out] tensor")
    wp, wn, keep = _workspace(TG_OP_LORA_UP, (T, d_out, r, 0), _DT[H.dtype], _DT[Y.dtype], ws, H.device)
    _check(lib().tg_lora_up_add(_ptr(H), _ptr(B), _ptr(Y), T, d_out, r, float(scale), _DT[H.dtype], _DT[Y.dtype],
                                wp, wn, _stream(stream)), "tg_lora_up_add")
    _keep(keep, stream)
    return Y
def tg_lora_grad(X, A, B, H, dY, out_dtype=None, want_dH=False, outs=None, ws=None, stream=None):
    """Gradients of Y = (X A^T) B^T: returns dict dA, dB, dX (and dH in FP32 when asked)."""
    for t, n in ((X, "X"), (A, "A"), (B, "B"), (H, "H"), (dY, "dY")):
        _need(t, n, 2)
    T, d_in = X.shape
    r = A.shape[0]
    d_out = B.shape[0]
    if A.shape[1] != d_in or B.shape[1] != r or H.shape != (T, r) or dY.shape != (T, d_out):
        raise ValueError("inconsistent LoRA shapes")
    od = out_dtype or X.dtype
    outs = dict(outs or {})
    dA = _out(outs.get("dA"), (r, d_in), od, X.device, "dA")
    dB = _out(outs.get("dB"), (d_out, r), od, X.device, "dB")
    dX = _out(outs.get("dX"), (T, d_in), od, X.device, "dX")
    dH = _out(outs.get("dH"), (T, r), torch.float32, X.device, "dH") if (want_dH or "dH" in outs) else None
    din = _DT[X.dtype]
    wp, wn, keep = _workspace(TG_OP_LORA_GRAD, (T, d_in, d_out, r), din, _DT[od], ws, X.device)
    _check(lib().tg_lora_grad(_ptr(X), _ptr(A), _ptr(B), _ptr(H), _ptr(dY), _ptr(dA), _ptr(dB), _ptr(dX),
                              _ptr(dH), T, d_in, d_out, r, din, _DT[od], wp, wn, _stream(stream)), "tg_lora_grad")
    _keep(keep, stream)
    res = {"dA": dA, "dB": dB, "dX": dX}
    if dH is not None:
        res["dH"] = dH
    return res


def tg_lora_grad_add(X, A, B, H, dY, dX, scale, want_dH=False, outs=None, ws=None, stream=None):
    """Gradients of Y = X W^T + scale (X A^T) B^T with the LoRA part added into
    dX (the base layer's dgrad on entry): returns dict dA, dB (scaled), dX (the
    same tensor, updated) and dH (FP32, unscaled) when asked.  dA and dB take
    dX's dtype."""
    for t, n in ((X, "X"), (A, "A"), (B, "B"), (H, "H"), (dY, "dY")):
        _need(t, n, 2)
    T, d_in = X.shape
    r = A.shape[0]
    d_out = B.shape[0]
    if A.shape[1] != d_in or B.shape[1] != r or H.shape != (T, r) or dY.shape != (T, d_out):
        raise ValueError("inconsistent LoRA shapes")
    if dX is None or tuple(dX.shape) != (T, d_in) or not dX.is_contiguous():
        raise ValueError("dX must be a contiguous [T, d_in] tensor")
    od = dX.dtype
    outs = dict(outs or {})
    dA = _out(outs.get("dA"), (r, d_in), od, X.device, "dA")
    dB = _out(outs.get("dB"), (d_out, r), od, X.device, "dB")
    dH = _out(outs.get("dH"), (T, r), torch.float32, X.device, "dH") if (want_dH or "dH" in outs) else None
    din = _DT[X.dtype]
    wp, wn, keep = _workspace(TG_OP_LORA_GRAD, (T, d_in, d_out, r), din, _DT[od], ws, X.device)
    _check(lib().tg_lora_grad_add(_ptr(X), _ptr(A), _ptr(B), _ptr(H), _ptr(dY), _ptr(dA), _ptr(dB), _ptr(dX),
                                  _ptr(dH), T, d_in, d_out, r, float(scale), din, _DT[od], wp, wn, _stream(stream)),
           "tg_lora_grad_add")
    _keep(keep, stream)
    res = {"dA": dA, "dB": dB, "dX": dX}
    if dH is not None:
        res["dH"] = dH
    return res


def _need_f32(t, name, shape):
    _need(t, name, len(shape))
    if t.dtype != torch.float32 or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be an FP32 {tuple(shape)} tensor, got {t.dtype} {tuple(t.shape)}")


def tg_lora_down_f32w(X, A, H=None, out_dtype=None, ws=None, stream=None):
    """H[T, r] = X[T, d_in] A[r, d_in]^T with an FP32 factor A and 16-bit X."""
    _need(X, "X", 2)
    T, d_in = X.shape
    r = A.shape[0]
    _need_f32(A, "A", (r, d_in))
    H = _out(H, (T, r), out_dtype or X.dtype, X.device, "H")
    wp, wn, keep = _workspace(TG_OP_LORA_DOWN_F32W, (T, d_in, r, 0), _DT[X.dtype], _DT[H.dtype], ws, X.device)
    _check(lib().tg_lora_down_f32w(_ptr(X), _ptr(A), _ptr(H), T, d_in, r, _DT[X.dtype], _DT[H.dtype], wp, wn,
                                   _stream(stream)), "tg_lora_down_f32w")
    _keep(keep, stream)
    return H


def tg_lora_up_f32w(H, B, Y=None, out_dtype=None, ws=None, stream=None):
    """Y[T, d_out] = H[T, r] B[d_out, r]^T with an FP32 factor B and 16-bit H."""
    _need(H, "H", 2)
    T, r = H.shape
    d_out = B.shape[0]
    _need_f32(B, "B", (d_out, r))
    Y = _out(Y, (T, d_out), out_dtype or H.dtype, H.device, "Y")
    wp, wn, keep = _workspace(TG_OP_LORA_UP_F32W, (T, d_out, r, 0), _DT[H.dtype], _DT[Y.dtype], ws, H.device)
    _check(lib().tg_lora_up_f32w(_ptr(H), _ptr(B), _ptr(Y), T, d_out, r, _DT[H.dtype], _DT[Y.dtype], wp, wn,
                                 _stream(stream)), "tg_lora_up_f32w")
    _keep(keep, stream)
    return Y


def tg_lora_grad_f32w(X, A, B, H, dY, out_dtype=None, want_dH=False, outs=None, ws=None, stream=None):
    """Gradients of Y = (X A^T) B^T with FP32 factors A, B and 16-bit X, H, dY:
    dict dA, dB (FP32), dX (out_dtype, default X's) and dH (FP32) when asked."""
    for t, n in ((X, "X"), (H, "H"), (dY, "dY")):
        _need(t, n, 2)
    T, d_in = X.shape
    r = A.shape[0]
    d_out = B.shape[0]
    _need_f32(A, "A", (r, d_in))
    _need_f32(B, "B", (d_out, r))
    if H.shape != (T, r) or dY.shape != (T, d_out):
        raise ValueError("inconsistent LoRA shapes")
    od = out_dtype or X.dtype
    outs = dict(outs or {})
    dA = _out(outs.get("dA"), (r, d_in), torch.float32, X.device, "dA")
    dB = _out(outs.get("dB"), (d_out, r), torch.float32, X.device, "dB")
    dX = _out(outs.get("dX"), (T, d_in), od, X.device, "dX")
    dH = _out(outs.get("dH"), (T, r), torch.float32, X.device, "dH") if (want_dH or "dH" in outs) else None
    din = _DT[X.dtype]
    wp, wn, keep = _workspace(TG_OP_LORA_GRAD_F32W, (T, d_in, d_out, r), din, _DT[od], ws, X.device)
    _check(lib().tg_lora_grad_f32w(_ptr(X), _ptr(A), _ptr(B), _ptr(H), _ptr(dY), _ptr(dA), _ptr(dB), _ptr(dX),
                                   _ptr(dH), T, d_in, d_out, r, din, _DT[od], wp, wn, _stream(stream)),
           "tg_lora_grad_f32w")
    _keep(keep, stream)
    res = {"dA": dA, "dB": dB, "dX": dX}
    if dH is not None:
        res["dH"] = dH
    return res


def tg_attn_fwd(Q, K, V, O=None, scale=None, out_dtype=None, stream=None):
    """Fused attention forward: O = softmax(scale Q K^T) V per head; Q, K, V [heads, s, 64]."""
    for t, n in ((Q, "Q"), (K, "K"), (V, "V")):
        _need(t, n, 3)
    heads, s, d = Q.shape
    if tuple(K.shape) != (heads, s, d) or tuple(V.shape) != (heads, s, d) or K.dtype != Q.dtype or V.dtype != Q.dtype:
        raise ValueError("K and V must match Q")
    O = _out(O, (heads, s, d), out_dtype or Q.dtype, Q.device, "O")
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(d)
    _check(lib().tg_attn_fwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), heads, s, d, sc, _DT[Q.dtype], _DT[O.dtype],
                             _stream(stream)), "tg_attn_fwd")
    return O


def tg_attn_bwd(Q, K, V, dO, scale=None, out_dtype=None, outs=None, ws=None, stream=None):
    """Fused attention backward: {"dQ", "dK", "dV"} of the forward of tg_attn_fwd given dO; all [heads, s, 64]."""
    for t, n in ((Q, "Q"), (K, "K"), (V, "V"), (dO, "dO")):
        _need(t, n, 3)
    heads, s, d = Q.shape
    for t in (K, V, dO):
        if tuple(t.shape) != (heads, s, d) or t.dtype != Q.dtype:
            raise ValueError("K, V and dO must match Q")
    outs = dict(outs or {})
    dt = out_dtype or (next(iter(outs.values())).dtype if outs else Q.dtype)
    res = {k: _out(outs.get(k), (heads, s, d), dt, Q.device, k) for k in ("dQ", "dK", "dV")}
    sc = float(scale) if scale is not None else 1.0 / math.sqrt(d)
    wptr, wbytes, buf = _workspace(TG_OP_ATTN_BWD, (heads, s, d, 0), _DT[Q.dtype], _DT[dt], ws, Q.device)
    _check(lib().tg_attn_bwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(dO), _ptr(res["dQ"]), _ptr(res["dK"]), _ptr(res["dV"]),
                             heads, s, d, sc, _DT[Q.dtype], _DT[dt], wptr, wbytes, _stream(stream)), "tg_attn_bwd")
    if buf is not ws:
        _keep(buf, stream)
    return res


def tg_bmm_attn(op, A, B, C=None, out_dtype=None, ws=None, stream=None):
    """One of the attention products (see include/tg.h); op is a name or a tg_attn_op value."""
    code = ATTN_OPS[op] if isinstance(op, str) else int(op)
    _need(A, "A", 3), _need(B, "B", 3)
    batch, s, d = B.shape
    ss_out = code in (0, 2)
    if code in (0, 2):
        if tuple(A.shape) != (batch, s, d):
            raise ValueError("A must be [batch, s, d]")
    elif tuple(A.shape) != (batch, s, s):
        raise ValueError("A must be [batch, s, s]")
    C = _out(C, (batch, s, s if ss_out else d), out_dtype or A.dtype, A.device, "C")
    wp, wn, keep = _workspace(TG_OP_BMM_ATTN, (code, batch, s, d), _DT[A.dtype], _DT[C.dtype], ws, A.device)
    _check(lib().tg_bmm_attn(code, _ptr(A), _ptr(B), _ptr(C), batch, s, d, _DT[A.dtype], _DT[C.dtype], wp, wn,
                             _stream(stream)), "tg_bmm_attn")
    _keep(keep, stream)
    return C


# The operators below are called many times a step on small tensors: their
# checks read each tensor's attributes once, and addresses go to ctypes as
# plain integers (0: NULL, for an empty tensor).
def _raw_stream(stream, device):
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """Memory that a call on `stream` (None: the current one) writes.  It is taken from that stream's: the current
    stream's may still be read by work queued there earlier, for which the other does not wait."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _new(shape, dtype, device, stream):
    """An output of a call on `stream`, for the caller to go on with on the current one."""
    t = _empty(shape, dtype, device, stream)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(device))
    return t


# Workspaces of calls on the current stream, kept by each host thread for each
# (device, stream): an allocation a call took a quarter of a small call's host
# time.  A thread's calls on one stream use its buffer one after the other.  Two
# threads never share one: a call is several launches that pass data through its
# workspace, and another thread's launches on the same stream may land between
# them.  As with any memory of torch's allocator, work on a stream made outside
# torch has to be finished before that stream is destroyed.  Not kept: large
# ones, those of a call that is being captured (a graph outlives them) and of a
# caller's own stream.
_kept = threading.local()
_KEEP_BYTES = 32 << 20


def _scratch(op, dims, din, dout, ws, device, stream, raw):
    """(address, bytes, buffer) of a call's workspace; raw: the stream's handle.  The caller holds the buffer until
    the call has returned: a kept one may be replaced meanwhile."""
    n = (_lib or lib()).tg_workspace_size(op, *dims, din, dout)
    if n == 0 or n == SIZE_MAX:  # SIZE_MAX: sizes or types that the call itself will refuse
        return 0, 0, None
    return _scratch_alloc(n, ws, device, stream, raw)


def _scratch_alloc(n, ws, device, stream, raw):
    if ws is not None and ws.numel() * ws.element_size() >= n:
        return ws.data_ptr(), ws.numel() * ws.element_size(), None
    if stream is not None or n > _KEEP_BYTES or torch.cuda.is_current_stream_capturing():
        buf = _empty(n, torch.uint8, device, stream)
        return buf.data_ptr(), n, buf
    kept = _kept.__dict__
    key = (device.index, raw)
    mine = kept.get(key)
    if mine is None or mine[1] < n:
        buf = torch.empty(max(n, 1 << 20), dtype=torch.uint8, device=device)
        mine = kept[key] = (buf.data_ptr(), buf.numel(), buf)
    return mine


def _like(t, name, shape, dtype, device):
    """Address of a tensor that must be contiguous with this shape, type and device."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on {device}")
    return t.data_ptr()


def _grouped(name, op, A, B, W_shape, offsets, rows, out_arg, out_shape, out_name, out_dtype, ws, stream):
    """A, B: the two operands as the C entry point takes them; W_shape: (E, d_out, d_in)."""
    E, d_out, d_in = W_shape
    dev, dt = A.device, A.dtype
    if B.device != dev:
        raise ValueError("the operands must be on one device")
    off = _like(offsets, "offsets", (E + 1,), torch.int32, dev)
    if out_arg is None:
        C = _new(out_shape, out_dtype or dt, dev, stream)
        c = C.data_ptr()
    else:
        C = out_arg
        c = _like(C, out_name, out_shape, out_dtype or getattr(C, "dtype", dt), dev)
    din, dout = _DT.get(dt, -1), _DT.get(C.dtype, -1)
    a, b = A.data_ptr(), B.data_ptr()
    raw = _raw_stream(stream, dev)
    wp, wn, held = _scratch(TG_OP_GROUPED_UNALIGNED if (a | b) & 15 else op, (rows, E, d_out, d_in), din, dout, ws, dev,
                            stream, raw)
    status = getattr(_lib or lib(), name)(a, b, off, c, rows, E, d_out, d_in, din, dout, wp, wn, raw)
    if status:
        raise TGError(status, name)
    return C


def tg_grouped_fwd(X, W, offsets, Y=None, out_dtype=None, ws=None, stream=None):
    """Y[t] = X[t] W[e]^T for the rows offsets[e] <= t < offsets[e + 1] of expert e, zeros in rows of no
    expert: X [T, d_in], W [E, d_out, d_in], offsets [E + 1] int32 on the device."""
    _need(X, "X", 2), _need(W, "W", 3)
    T, d_in = X.shape
    E, d_out, k = W.shape
    if k != d_in or W.dtype != X.dtype:
        raise ValueError("W must be [E, d_out, d_in] with X's dtype")
    return _grouped("tg_grouped_fwd", TG_OP_GROUPED_FWD, X, W, (E, d_out, d_in), offsets, T, Y, (T, d_out), "Y",
                    out_dtype, ws, stream)


def tg_grouped_dgrad(dY, W, offsets, dX=None, out_dtype=None, ws=None, stream=None):
    """dX[t] = dY[t] W[e] for the rows of expert e, zeros in rows of no expert: dY [T, d_out],
    W [E, d_out, d_in], offsets [E + 1] int32 on the device."""
    _need(dY, "dY", 2), _need(W, "W", 3)
    T, d_out = dY.shape
    E, k, d_in = W.shape
    if k != d_out or W.dtype != dY.dtype:
        raise ValueError("W must be [E, d_out, d_in] with dY's dtype")
    return _grouped("tg_grouped_dgrad", TG_OP_GROUPED_DGRAD, dY, W, (E, d_out, d_in), offsets, T, dX, (T, d_in), "dX",
                    out_dtype, ws, stream)


def tg_grouped_wgrad(dY, X, offsets, dW=None, out_dtype=None, ws=None, stream=None):
    """dW[e] = sum over the rows t of expert e of dY[t]^T X[t] (zeros for an expert without rows):
    dY [T, d_out], X [T, d_in], offsets [E + 1] int32 on the device; dW [E, d_out, d_in]."""
    _need(dY, "dY", 2), _need(X, "X", 2)
    T, d_out = dY.shape
    if X.shape[0] != T or X.dtype != dY.dtype:
        raise ValueError("X must be [T, d_in] with dY's dtype")
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be a 1-d tensor of E + 1 values")
    shape = (offsets.shape[0] - 1, d_out, X.shape[1])
    return _grouped("tg_grouped_wgrad", TG_OP_GROUPED_WGRAD, dY, X, shape, offsets, T, dW, shape, "dW", out_dtype, ws,
                    stream)


def _gate(gate, T, d, dtype, device):
    """(kind, shape, address) of a gate."""
    if gate is None:
        return TG_GATE_NONE, None, 0
    shape = tuple(gate.shape)
    kind = TG_GATE_CHANNEL if shape == (d,) else TG_GATE_TOKEN if shape == (T, 1) else TG_GATE_FULL
    if kind == TG_GATE_FULL and shape != (T, d):
        raise ValueError("gate must be [d], [T, 1] or [T, d]")
    return kind, shape, _like(gate, "gate", shape, dtype, device)


def _result(res, outs, name, shape, dtype, device, stream):
    """Address of an output: the caller's, or a new one; kept in res."""
    t = outs.get(name) if outs else None
    if t is None:
        t = res[name] = _new(shape, dtype, device, stream)
        return t.data_ptr()
    res[name] = t
    return _like(t, name, shape, dtype, device)


def _stream_type(H, name, dtype):
    rt = getattr(H, "dtype", None)
    if rt is not dtype and rt is not torch.float32:
        raise ValueError(f"{name} must have B's dtype or FP32")
    return rt


def tg_norm_residual_fwd(B, H, w_post, w_pre, gate=None, res_scale=1.0, eps=1e-6, outs=None, stream=None):
    """u = B rstd_b w_post, H_out = res_scale H + gate u, N = H_out rstd_h w_pre with rstd = (mean square + eps)^-1/2
    over the row: B, H [T, d], w_post, w_pre [d], gate None, [d], [T, 1] or [T, d].  H may be FP32 beside 16-bit B.
    Returns {"H", "N", "rstd_b", "rstd_h"} (outs may give any of them; outs["H"] may be H)."""
    _need(B, "B", 2)
    T, d = shape = tuple(B.shape)
    dev, dt = B.device, B.dtype
    rt = _stream_type(H, "H", dt)
    h = _like(H, "H", shape, rt, dev)
    wq, wp = _like(w_post, "w_post", (d,), dt, dev), _like(w_pre, "w_pre", (d,), dt, dev)
    kind, _, g = _gate(gate, T, d, dt, dev)
    res = {}
    ho, n = _result(res, outs, "H", shape, rt, dev, stream), _result(res, outs, "N", shape, dt, dev, stream)
    rb, rh = (_result(res, outs, k, (T,), torch.float32, dev, stream) for k in ("rstd_b", "rstd_h"))
    status = (_lib or lib()).tg_norm_residual_fwd(B.data_ptr(), h, wq, wp, g, kind, ho, n, rb, rh, T, d, res_scale, eps,
                                                  _DT.get(dt, -1), _DT[rt] if rt in _DT else -1,
                                                  _raw_stream(stream, dev))
    if status:
        raise TGError(status, "tg_norm_residual_fwd")
    return res


def tg_norm_residual_bwd(dH_out, dN, B, H_out, w_post, w_pre, rstd_b, rstd_h, gate=None, res_scale=1.0, out_dtype=None,
                         outs=None, ws=None, stream=None):
    """Gradients of <dH_out, H_out> + <dN, N> for the forward of tg_norm_residual_fwd: {"dB", "dH", "dw_post",
    "dw_pre"} and "dgate" when there is a gate.  out_dtype (B's dtype or FP32; by default that of those in outs):
    dw_post, dw_pre and the gradient of a broadcast gate.  outs may give any of them."""
    _need(B, "B", 2)
    T, d = shape = tuple(B.shape)
    dev, dt = B.device, B.dtype
    rt = _stream_type(H_out, "H_out", dt)
    f32 = torch.float32
    ho, dho = _like(H_out, "H_out", shape, rt, dev), _like(dH_out, "dH_out", shape, rt, dev)
    dn = _like(dN, "dN", shape, dt, dev)
    wq, wp = _like(w_post, "w_post", (d,), dt, dev), _like(w_pre, "w_pre", (d,), dt, dev)
    rb, rh = _like(rstd_b, "rstd_b", (T,), f32, dev), _like(rstd_h, "rstd_h", (T,), f32, dev)
    kind, gshape, g = _gate(gate, T, d, dt, dev)
    ot = out_dtype
    if ot is None:  # that of any output of this type that is given
        ot = dt
        for k in ("dw_post", "dw_pre", "dgate") if outs else ():
            t = outs.get(k)
            if t is not None and (k != "dgate" or kind in (TG_GATE_CHANNEL, TG_GATE_TOKEN)):
                ot = t.dtype
                break
    res = {}
    db, dh = _result(res, outs, "dB", shape, dt, dev, stream), _result(res, outs, "dH", shape, rt, dev, stream)
    dwq, dwp = _result(res, outs, "dw_post", (d,), ot, dev, stream), _result(res, outs, "dw_pre", (d,), ot, dev, stream)
    gt = dt if kind == TG_GATE_FULL else ot
    dg = 0 if kind == TG_GATE_NONE else _result(res, outs, "dgate", gshape, gt, dev, stream)
    din, dout = _DT.get(dt, -1), _DT.get(ot, -1)
    raw = _raw_stream(stream, dev)
    wsp, wsn, held = _scratch(TG_OP_NORM_RESIDUAL_BWD, (T, d, 0, 0), din, dout, ws, dev, stream, raw)
    status = (_lib or lib()).tg_norm_residual_bwd(dho, dn, B.data_ptr(), ho, wq, wp, g, kind, rb, rh, db, dh, dwq, dwp,
                                                  dg, T, d, res_scale, din, _DT.get(rt, -1), dout, wsp, wsn, raw)
    if status:
        raise TGError(status, "tg_norm_residual_bwd")
    return res


class TGTensorList:
    """Addresses, sizes and types of tensors, laid out once for tg_grad_norm and tg_grad_clip.  Keeps the
    tensors and their memory alive; they must not be resized while it is used.  A call on a list with a tensor
    that was given other memory since is refused."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        for k, t in enumerate(self.tensors):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous() or t.dtype not in _DT:
                raise ValueError(f"tensor {k} must be a contiguous bf16, fp16 or FP32 CUDA tensor")
            if t.device != self.tensors[0].device:
                raise ValueError("the tensors must be on one device")
        n = len(self.tensors)
        self.device = self.tensors[0].device if n else None
        self._addresses = [t.data_ptr() for t in self.tensors]
        self._memory = [t.untyped_storage() for t in self.tensors]  # until the list goes, nothing else gets it
        self._arrays = ((ctypes.c_void_p * n)(*[a if t.numel() else 0 for a, t in zip(self._addresses, self.tensors)]),
                        (ctypes.c_int64 * n)(*[t.numel() for t in self.tensors]),
                        (ctypes.c_int32 * n)(*[_DT[t.dtype] for t in self.tensors]))
        self.pointers, self.numels, self.dtypes = (ctypes.addressof(a) for a in self._arrays)
        self.kinds = bytes(self._arrays[1]) + bytes(self._arrays[2])

    def _check(self):
        now = list(map(torch.Tensor.data_ptr, self.tensors))
        if now != self._addresses:
            k = next((k for k, (a, b) in enumerate(zip(now, self._addresses)) if a != b), len(self._addresses))
            raise ValueError(f"tensor {k} has other memory than when the list was laid out: lay it out again")

    def __len__(self):
        return len(self.tensors)

    def __iter__(self):
        return iter(self.tensors)


def tg_tensor_list(tensors) -> TGTensorList:
    """A list of gradient tensors to hand to tg_grad_norm and tg_grad_clip step after step."""
    return tensors if isinstance(tensors, TGTensorList) else TGTensorList(tensors)


def _laid_out(tensors):
    if not isinstance(tensors, TGTensorList):
        return TGTensorList(tensors)
    tensors._check()  # 80 ns a tensor: two lists of 56 take 9 us of a call
    return tensors


def _grads(name, grads, outs, max_norm, norm, ws, stream):
    g = _laid_out(grads)
    o = g if outs is None else _laid_out(outs)
    if o is not g and (o.kinds != g.kinds or o.device != g.device):
        raise ValueError("outs must match the gradients' sizes and dtypes one by one, on their device")
    n = len(g.tensors)
    dev = g.device
    if dev is None:
        dev = norm.device if norm is not None else torch.device("cuda", torch.cuda.current_device())
    if norm is None:
        norm = _new(1, torch.float32, dev, stream)
    at = _like(norm, "norm", (1,), torch.float32, dev)
    s = _raw_stream(stream, dev)
    wp, wn, held = _scratch(TG_OP_GRAD_CLIP, (n, 0, 0, 0), TG_F32, TG_F32, ws, dev, stream, s)
    if name == "tg_grad_norm":
        status = (_lib or lib()).tg_grad_norm(g.pointers, g.numels, g.dtypes, n, at, wp, wn, s)
    else:
        status = (_lib or lib()).tg_grad_clip(g.pointers, o.pointers, g.numels, g.dtypes, n, max_norm, at, wp, wn, s)
    if status:
        raise TGError(status, name)
    return norm


def tg_grad_norm(grads, norm=None, ws=None, stream=None):
    """The L2 norm of all the tensors' elements together, as one FP32 value on the device ([1])."""
    return _grads("tg_grad_norm", grads, None, 0.0, norm, ws, stream)


def tg_grad_clip(grads, max_norm, outs=None, norm=None, ws=None, stream=None):
    """Scale every tensor by min(1, max_norm / (norm + 1e-6)), norm the L2 norm of all their elements together:
    in place, or into outs (tensors of the same types and sizes).  grads and outs: tensors, or lists laid out
    once with tg_tensor_list.  Returns the norm (before scaling), one FP32 value on the device ([1])."""
    return _grads("tg_grad_clip", grads, outs, max_norm, norm, ws, stream)


# The operators below take few microseconds on the GPU: their checks are written out, each attribute read once.
_Tensor = torch.Tensor
_current_device = torch._C._cuda_getDevice


def _on_current(t, name, ndim):
    """A contiguous CUDA tensor on the current device; returns its device and type."""
    _need(t, name, ndim)
    if t.get_device() != _current_device():
        raise ValueError(f"{name} must be on the current device")
    return t.device, t.dtype


def _at(t, name, shape, dtype, index):
    """Address of a tensor that must be contiguous with this shape, type and CUDA device (as _like)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:  # not a tensor
        pass
    raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on cuda:{index}")


@functools.lru_cache(maxsize=1024)
def _ws_bytes(device_index, op, d0, d1, d2, din, dout):
    """tg_workspace_size on the current device, whose index is in the key."""
    return lib().tg_workspace_size(op, d0, d1, d2, 0, din, dout)


def _scratch_of(n, ws, device, stream, raw):
    """As _scratch, for a workspace of n bytes."""
    if n == 0 or n == SIZE_MAX:  # SIZE_MAX: sizes or types that the call itself will refuse
        return 0, 0, None
    if ws is None and stream is None and n <= _KEEP_BYTES:
        mine = _kept.__dict__.get((device.index, raw))
        if mine is not None and mine[1] >= n and not torch._C._cuda_isCurrentStreamCapturing():
            return mine
    return _scratch_alloc(n, ws, device, stream, raw)


def tg_layer_norm_fwd(X, w, b=None, eps=1e-5, outs=None, stream=None):
    """Y = (X - mean) rstd w + b over the rows of X [T, d], rstd = (variance + eps)^-1/2; w, b [d].
    Returns {"Y", "mean", "rstd"} (outs may give any of them; outs["Y"] may be X)."""
    dev, dt = _on_current(X, "X", 2)
    index = dev.index
    shape = X.shape
    T, d = shape
    wp = _at(w, "w", (d,), dt, index)
    bp = 0 if b is None else _at(b, "b", (d,), dt, index)
    o = outs or {}
    Y, mean, rstd = o.get("Y"), o.get("mean"), o.get("rstd")
    if Y is None:
        Y = _new(shape, dt, dev, stream)
    if mean is None:
        mean = _new((T,), torch.float32, dev, stream)
    if rstd is None:
        rstd = _new((T,), torch.float32, dev, stream)
    f32 = torch.float32
    status = (_lib or lib()).tg_layer_norm_fwd(X.data_ptr(), wp, bp, _at(Y, "Y", shape, dt, index),
                                               _at(mean, "mean", (T,), f32, index), _at(rstd, "rstd", (T,), f32, index), T, d,
                                               eps, _DT.get(dt, -1), _raw_stream(stream, dev))
    if status:
        raise TGError(status, "tg_layer_norm_fwd")
    return {"Y": Y, "mean": mean, "rstd": rstd}


def tg_layer_norm_bwd(dY, X, w, mean, rstd, dR=None, bias=True, out_dtype=None, outs=None, ws=None, stream=None):
    """Gradients of <dY, Y> for the forward of tg_layer_norm_fwd: {"dX", "dw"} and, with `bias`, "db".  dR [T, d]: a
    gradient to add to dX.  out_dtype (X's dtype or FP32; by default that of those in outs): dw and db."""
    dev, dt = _on_current(X, "X", 2)
    index = dev.index
    shape = X.shape
    T, d = shape
    f32 = torch.float32
    o = outs or {}
    dX, dw, db = o.get("dX"), o.get("dw"), o.get("db") if bias else None
    ot = out_dtype
    if ot is None:  # that of either output that is given
        ot = getattr(dw if dw is not None else db, "dtype", dt)
    if dX is None:
        dX = _new(shape, dt, dev, stream)
    if dw is None:
        dw = _new((d,), ot, dev, stream)
    if bias and db is None:
        db = _new((d,), ot, dev, stream)
    din, dout = _DT.get(dt, -1), _DT.get(ot, -1)
    raw = _raw_stream(stream, dev)
    wsp, wsn, held = _scratch_of(_ws_bytes(index, TG_OP_LAYER_NORM_BWD, T, d, 0, din, dout), ws, dev, stream, raw)
    status = (_lib or lib()).tg_layer_norm_bwd(
        _at(dY, "dY", shape, dt, index), X.data_ptr(), _at(w, "w", (d,), dt, index), _at(mean, "mean", (T,), f32, index),
        _at(rstd, "rstd", (T,), f32, index), 0 if dR is None else _at(dR, "dR", shape, dt, index), _at(dX, "dX", shape, dt, index),
        _at(dw, "dw", (d,), ot, index), _at(db, "db", (d,), ot, index) if bias else 0, T, d, din, dout, wsp, wsn, raw)
    if status:
        raise TGError(status, "tg_layer_norm_bwd")
    return {"dX": dX, "dw": dw, "db": db} if bias else {"dX": dX, "dw": dw}


def _act(act):
    code = ACTS.get(act) if isinstance(act, str) else act
    if code not in (0, 1, 2, 3):
        raise ValueError(f"act must be one of {', '.join(ACTS)}")
    return code


def tg_gated_fwd(X, W, act="silu", keep=False, outs=None, ws=None, stream=None):
    """[G U] = X W^T and H = act(G) U in one kernel: X [T, d], W [2 f, d] (gate rows, then up rows).  Returns {"H"}
    and, with `keep`, "GU" [T, 2 f], which the backward takes.  act: silu, gelu, gelu_tanh or relu."""
    dev, dt = _on_current(X, "X", 2)
    index = dev.index
    T, d = X.shape
    rows = W.shape[0] if isinstance(W, _Tensor) and W.dim() == 2 else 0
    if rows % 2:
        raise ValueError("W must have an even number of rows: the gate's, then the up projection's")
    f = rows // 2
    wp = _at(W, "W", (rows, d), dt, index)
    a = _act(act)
    o = outs or {}
    H, GU = o.get("H"), o.get("GU") if keep else None
    if H is None:
        H = _new((T, f), dt, dev, stream)
    if keep and GU is None:
        GU = _new((T, rows), dt, dev, stream)
    din = _DT.get(dt, -1)
    x = X.data_ptr()
    raw = _raw_stream(stream, dev)
    n = _ws_bytes(index, TG_OP_GATED_UNALIGNED if (x | wp) & 15 else TG_OP_GATED_FWD, T, f, d, din, din)
    wsp, wsn, held = _scratch_of(n, ws, dev, stream, raw)
    status = (_lib or lib()).tg_gated_fwd(x, wp, _at(H, "H", (T, f), dt, index), _at(GU, "GU", (T, rows), dt, index) if keep else 0,
                                          T, f, d, a, din, wsp, wsn, raw)
    if status:
        raise TGError(status, "tg_gated_fwd")
    return {"H": H, "GU": GU} if keep else {"H": H}


def tg_gated_bwd(dY, W_down, GU, act="silu", keep=False, outs=None, ws=None, stream=None):
    """Through the down projection and the gate: with dH = dY W_down (never stored), dGU = [dH U act'(G), dH act(G)];
    dY [T, d], W_down [d, f], GU [T, 2 f] of the forward.  Returns {"dGU"} and, with `keep`, "H" = act(G) U for the
    down projection's weight gradient (outs may give them; outs["dGU"] may be GU)."""
    dev, dt = _on_current(dY, "dY", 2)
    index = dev.index
    T, d = dY.shape
    f = W_down.shape[1] if isinstance(W_down, _Tensor) and W_down.dim() == 2 else 0
    wp = _at(W_down, "W_down", (d, f), dt, index)
    two = (T, 2 * f)
    gp = _at(GU, "GU", two, dt, index)
    a = _act(act)
    o = outs or {}
    dGU, H = o.get("dGU"), o.get("H") if keep else None
    if dGU is None:
        dGU = _new(two, dt, dev, stream)
    if keep and H is None:
        H = _new((T, f), dt, dev, stream)
    din = _DT.get(dt, -1)
    y = dY.data_ptr()
    raw = _raw_stream(stream, dev)
    n = _ws_bytes(index, TG_OP_GATED_UNALIGNED if (y | wp) & 15 else TG_OP_GATED_BWD, T, f, d, din, din)
    wsp, wsn, held = _scratch_of(n, ws, dev, stream, raw)
    status = (_lib or lib()).tg_gated_bwd(y, wp, gp, _at(dGU, "dGU", two, dt, index), _at(H, "H", (T, f), dt, index) if keep else 0,
                                          T, f, d, a, din, wsp, wsn, raw)
    if status:
        raise TGError(status, "tg_gated_bwd")
    return {"dGU": dGU, "H": H} if keep else {"dGU": dGU}


# (a, b, c) of s -> a s + b s^3 + c s^5: five of them take every singular value into about [0.7, 1.2]
ORTH_QUINTIC = (3.4445, -4.7750, 2.0315)


@functools.lru_cache(maxsize=64)
def _orth_coeffs(coeffs, steps):
    """(host array, steps) of one triple for all steps or of a triple for each."""
    one = bool(coeffs) and not any(isinstance(c, tuple) for c in coeffs)
    n = (5 if one else len(coeffs)) if steps is None else steps
    triples = (coeffs,) if one else coeffs
    if len(triples) != (1 if one else n) or not triples or any(not isinstance(c, tuple) or len(c) != 3 for c in triples):
        raise ValueError("coeffs must be (a, b, c), or such a triple for each step")
    if n != int(n) or not 1 <= n <= 64:
        raise ValueError("steps must be an integer from 1 to 64")
    flat = [x for c in triples for x in c]
    flat = flat * int(n) if one else flat
    return (ctypes.c_double * len(flat))(*flat), int(n)


def tg_orthogonalize(G, O=None, out_dtype=None, steps=None, coeffs=ORTH_QUINTIC, scale=1.0, eps=1e-7, ws=None, stream=None):
    """scale times the matrix (or each of a batch: G [rows, cols] or [batch, rows, cols]) that Newton-Schulz steps
    X <- a X + (b A + c A A) X, A = X X^T, make of X = G / (|G| + eps): close to the nearest one with orthonormal rows
    or columns.  coeffs: (a, b, c) for all steps (5 by default) or a triple for each.  G may be FP32; O is bf16 or
    fp16 (by default G's dtype, bf16 for FP32) and may be G."""
    if not isinstance(G, torch.Tensor) or G.dim() not in (2, 3):
        raise ValueError("G must be [rows, cols] or [batch, rows, cols]")
    dev, dt = _on_current(G, "G", G.dim())
    index = dev.index
    shape = tuple(G.shape)
    batch, rows, cols = shape if len(shape) == 3 else (1, *shape)
    array, n = _orth_coeffs(tuple(tuple(map(float, c)) if isinstance(c, (list, tuple)) else float(c) for c in coeffs), steps)
    ot = out_dtype or (O.dtype if O is not None else torch.bfloat16 if dt is torch.float32 else dt)
    if O is None:
        O = _new(shape, ot, dev, stream)
        o = O.data_ptr()
    else:
        o = _at(O, "O", shape, ot, index)
    din, dout = _DT.get(dt, -1), _DT.get(ot, -1)
    raw = _raw_stream(stream, dev)
    n_ws = _ws_bytes(index, TG_OP_ORTHOGONALIZE, batch, rows, cols, din, dout)
    wsp, wsn, held = _scratch_of(n_ws, ws, dev, stream, raw)
    status = (_lib or lib()).tg_orthogonalize(G.data_ptr(), o, batch, rows, cols, ctypes.addressof(array), n, scale, eps,
                                              din, dout, wsp, wsn, raw)
    if status:
        raise TGError(status, "tg_orthogonalize")
    return O


def tg_workspace_size(op, d0, d1, d2, d3, din, dout) -> int:
    return lib().tg_workspace_size(op, d0, d1, d2, d3, _DT.get(din, din), _DT.get(dout, dout))


def tg_stream_status(stream=None) -> int:
    return lib().tg_stream_status(_stream(stream))


def tg_status_string(status: int) -> str:
    return lib().tg_status_string(status).decode()


def tg_load_table(path) -> int:
    return lib().tg_load_table(None if path is None else str(path).encode())


def tg_version() -> int:
    return lib().tg_version()


def tg_plan_describe(op, M, N, K, batch, din, dout, sms) -> str:
    """The plan the tensor-core path would use (host only; see include/tg.h)."""
    buf = ctypes.create_string_buffer(512)
    n = lib().tg_plan_describe(op, M, N, K, batch, _DT[din], _DT[dout], sms, buf, 512)
    return buf.value.decode() if n else ""


def tg_last_call() -> str:
    buf = ctypes.create_string_buffer(512)
    lib().tg_last_call(buf, 512)
    return buf.value.decode()


def tg_wait_probe(timeout_us: int, stream=None) -> int:
    return lib().tg_wait_probe(timeout_us, _stream(stream))
