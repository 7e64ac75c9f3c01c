"""RMS norm with the residual's addition (include/gemm.h).

    y = rms_norm(x, weight)                          # x: R x K, float16 or bfloat16
    y, h = rms_norm(x, weight, residual)             # h = x + residual, y of h
    q, scale, h = rms_norm_i8(x, weight, residual)   # y as int8 rows: operands of i8.i8_matmul

`rms_norm` has gradients for x, residual and weight.  Argument marshalling only:
the work runs in libgemm.so's HIP kernels.
"""
import ctypes

import torch

from . import GEMM_BF16, GEMM_F16, GEMM_F32, _check, gemm_norm_problem, lib
from .grouped import NORM, NORM_I8, _need_gpu, _on_stream, _raw_stream, _remembered, _row_operator

_CODES = {torch.float16: GEMM_F16, torch.bfloat16: GEMM_BF16, torch.float32: GEMM_F32}


def gemm_rms_norm(problem, x, r, w, h, y, rstd=None, stream=None):
    """Device addresses (integers or None) and a hipStream_t (or None)."""
    _check(lib().gemm_rms_norm(ctypes.byref(problem), x, r, w, h, y, rstd, stream))


def gemm_rms_norm_i8(problem, x, r, w, h, q, scale, stream=None):
    """Device addresses (integers or None) and a hipStream_t (or None)."""
    _check(lib().gemm_rms_norm_i8(ctypes.byref(problem), x, r, w, h, q, scale, stream))


def gemm_rms_norm_grad_workspace(problem):
    n = ctypes.c_size_t()
    _check(lib().gemm_rms_norm_grad_workspace(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def gemm_rms_norm_grad(problem, dy, dh, h, w, rstd, dx, dw, workspace=None, workspace_bytes=0, stream=None):
    """Device addresses (integers or None) and a hipStream_t (or None)."""
    _check(lib().gemm_rms_norm_grad(ctypes.byref(problem), dy, dh, h, w, rstd, dx, dw, workspace, workspace_bytes, stream))


# ---------------------------------------------------------------- torch convenience

def _rows_arg(name, t, like=None):
    """A matrix of 16-bit rows, of the shape and type of `like`."""
    if like is None:
        if t.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("%s must be float16 or bfloat16, got %s" % (name, t.dtype))
        if t.dim() != 2:
            raise ValueError("%s must be 2-D, got %s" % (name, tuple(t.shape)))
    else:
        if t.dtype != like.dtype:
            raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, like.dtype))
        if t.shape != like.shape:
            raise ValueError("%s must be %s, got %s" % (name, tuple(like.shape), tuple(t.shape)))
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must have unit stride along its rows" % name)


def _arguments(x, weight, residual):
    _rows_arg("x", x)
    if residual is not None:
        _rows_arg("residual", residual, x)
    if weight.dtype not in (x.dtype, torch.float32):
        raise TypeError("weight has dtype %s, expected %s or float32" % (weight.dtype, x.dtype))
    if tuple(weight.shape) != (x.shape[1],) or (weight.shape[0] > 1 and weight.stride(0) != 1):
        raise ValueError("weight must be %d contiguous values, got %s" % (x.shape[1], tuple(weight.shape)))
    _need_gpu(x.device, ("x", x), ("weight", weight), ("residual", residual))


def _address(t):
    return t.data_ptr() if t is not None else None


def rms_norm_grad(dy, h, weight, rstd, dh=None, need_weight=True):
    """(dx, dw): the gradients of rms_norm for dy and, as the output of a residual's
    addition, dh, from the stream h that was normalized and its reciprocal root
    mean squares (float32, one per row).  dx is x's and the residual's; dw is None
    without need_weight."""
    _rows_arg("h", h)
    _rows_arg("dy", dy, h)
    if dh is not None:
        _rows_arg("dh", dh, h)
    _arguments(h, weight, None)
    if rstd.dtype != torch.float32 or tuple(rstd.shape) != (h.shape[0],) or (h.shape[0] > 1 and rstd.stride(0) != 1):
        raise ValueError("rstd must be %d contiguous float32 values" % h.shape[0])
    _need_gpu(h.device, ("dy", dy), ("dh", dh), ("rstd", rstd))

    def call():
        dx = torch.empty(h.shape, dtype=h.dtype, device=h.device)
        p = gemm_norm_problem()
        p.R, p.K = h.shape
        p.sx, p.sy, p.sh = dx.stride(0), dy.stride(0), h.stride(0)
        if dh is not None:
            p.sr, p.has_residual = dh.stride(0), 1
        p.dtype, p.weight, p.eps = _CODES[h.dtype], _CODES[weight.dtype], 1.0   # eps is in rstd
        dw, ws, need = None, None, 0
        if need_weight:
            dw = torch.empty(weight.shape, dtype=weight.dtype, device=h.device)
            need = gemm_rms_norm_grad_workspace(p)
            ws = torch.empty(need, dtype=torch.uint8, device=h.device) if need else None
        gemm_rms_norm_grad(p, dy.data_ptr(), _address(dh), h.data_ptr(), weight.data_ptr(), rstd.data_ptr(), dx.data_ptr(),
                           _address(dw), _address(ws), need, _raw_stream(h.device.index))
        return dx, dw
    return _on_stream(call, h.device, None, ())


def rms_norm(x, weight, residual=None, eps=1e-6, stream=None):
    """y[i] = h[i] weight / sqrt(mean(h[i]^2) + eps) with h = x, or, with a
    residual, h = x + residual rounded to their type; returns y, or (y, h).

    x, residual: R x K, float16 or bfloat16, unit stride along the rows; weight: K
    values of that type or float32.  Sums in float32, y rounded once.
    Differentiable (once, and in reverse mode: a forward-mode dual is refused); in a
    graph's capture that is refused while a graph of the same leaf that was recorded
    on the default stream is alive.  Asynchronous on `stream` (default: torch's
    current stream)."""
    eps = float(eps)
    if stream is None:
        out = _remembered(NORM, eps, x, weight, residual)
        if out is not None:
            return out
    _arguments(x, weight, residual)
    return _on_stream(lambda: _row_operator("norm", NORM, stream is None, eps, x, weight, residual), x.device, stream,
                      (x, weight, residual))


def rms_norm_i8(x, weight, residual=None, eps=1e-6, stream=None):
    """rms_norm's values in 8 bits: (q, scale), or (q, scale, h) with a residual.
    q: R x K int8, scale: R float32 as i8.i8_quantize makes them, of the values
    before any rounding to 16 bits.  No gradients: h, too, is without one."""
    eps = float(eps)
    if stream is None:
        out = _remembered(NORM_I8, eps, x, weight, residual)
        if out is not None:
            return out
    _arguments(x, weight, residual)
    return _on_stream(lambda: _row_operator("norm_i8", NORM_I8, stream is None, eps, x, weight, residual), x.device, stream,
                      (x, weight, residual))
