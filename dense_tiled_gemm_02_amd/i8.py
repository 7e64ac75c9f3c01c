"""Products of int8 rows with a scale for each, and the rows (include/gemm.h).

    w, w_scale = i8_quantize(W)                        # N x K weights, once: a scale per channel
    x, x_scale = i8_quantize(X)                        # M x K activations: a scale per token
    Y = i8_matmul(x, x_scale, w, w_scale, bias)        # about X W^T + bias

`norm.rms_norm_i8` makes x and x_scale from a stream that is normalized first.
Argument marshalling only: the work runs in libgemm.so's HIP kernels.
"""
import ctypes
import threading

import torch

from . import GEMM_BF16, GEMM_F16, GEMM_F32, _check, _keep_plan, _p, gemm_i8_problem, lib
from .grouped import I8, I8_ROWS, _need_gpu, _on_stream, _raw_stream, _remember, _remembered, _row_operator, _written
from .norm import _rows_arg

_CODES = {torch.float16: GEMM_F16, torch.bfloat16: GEMM_BF16, torch.float32: GEMM_F32}


class I8Plan:
    """Owns one gemm_i8_plan*; destroyed with the object."""

    def __init__(self, handle, problem):
        self.handle = handle
        self.problem = problem

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            lib().gemm_i8_plan_destroy(h)

    def describe(self):
        buf = ctypes.create_string_buffer(1024)
        _check(lib().gemm_i8_plan_describe(self.handle, buf, len(buf)))
        return buf.value.decode()


def gemm_i8_plan_create(problem, device=0):
    h = _p()
    _check(lib().gemm_i8_plan_create(ctypes.byref(problem), device, ctypes.byref(h)))
    return I8Plan(h, problem)


def gemm_i8_plan_create_for(problem, info):
    h = _p()
    _check(lib().gemm_i8_plan_create_for(ctypes.byref(problem), ctypes.byref(info), ctypes.byref(h)))
    return I8Plan(h, problem)


def gemm_i8_run(plan, X, x_scale, W, w_scale, bias, Y, stream=None):
    """Device addresses (integers or None) and a hipStream_t (or None)."""
    _check(lib().gemm_i8_run(plan.handle, X, x_scale, W, w_scale, bias, Y, stream))


def gemm_i8_quantize(x, dtype, R, K, sx, q, sq, scale, stream=None):
    """Device addresses (integers or None) and a hipStream_t (or None)."""
    _check(lib().gemm_i8_quantize(x, dtype, R, K, sx, q, sq, scale, stream))


# ---------------------------------------------------------------- torch convenience

_plans = {}
_lock = threading.Lock()   # guards _plans


def i8_quantize(X, stream=None):
    """(q, scale): each row of X (R x K, float16 or bfloat16, unit stride along the
    rows) as int8 steps of its own float32 scale, its largest magnitude / 127, so
    that X[i] is about q[i] scale[i]: activations with a scale per token, or a
    weight (N x K) with one per channel.  A row of zeros has the scale 0, a row
    with an infinity or a NaN the scale NaN.  No gradients.  Asynchronous on
    `stream` (default: torch's current stream)."""
    if stream is None:
        pair = _remembered(I8_ROWS, None, X)
        if pair is not None:
            return pair
    _rows_arg("X", X)
    _need_gpu(X.device, ("X", X))
    return _on_stream(lambda: _row_operator("i8_rows", I8_ROWS, stream is None, None, X), X.device, stream, (X,))


def _vector_arg(name, t, n, dtype):
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if tuple(t.shape) != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be %d contiguous values, got %s" % (name, n, tuple(t.shape)))


def i8_matmul(X, x_scale, W, w_scale, bias=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """Y[m, n] = (sum_k X[m, k] W[n, k]) x_scale[m] w_scale[n] (+ bias[n]).

    X: M x K int8, W: N x K int8 (unit stride along the rows, K below 2^17);
    x_scale, w_scale: M and N float32 values; bias: N values of the output's type;
    out_dtype: float16, bfloat16 or float32 (out's type where out is given).  The
    sums are exact; the scales and the bias are applied in float32, with one
    rounding to the output's type.  No gradients.  Asynchronous on `stream`
    (default: torch's current stream)."""
    plain = out is None and stream is None
    if plain:
        Y = _remembered(I8, out_dtype, X, x_scale, W, w_scale, bias)
        if Y is not None:
            return Y
    dtype = out_dtype if out is None else out.dtype
    if X.dtype != torch.int8 or W.dtype != torch.int8:
        raise TypeError("X and W must be int8, got %s and %s" % (X.dtype, W.dtype))
    if dtype not in _CODES:
        raise TypeError("the output is float16, bfloat16 or float32, got %s" % dtype)
    if X.dim() != 2 or W.dim() != 2 or X.shape[1] != W.shape[1]:
        raise ValueError("X and W must be M x K and N x K, got %s and %s" % (tuple(X.shape), tuple(W.shape)))
    (M, K), N = X.shape, W.shape[0]
    for name, t in (("X", X), ("W", W)):
        if K > 1 and t.stride(1) != 1:
            raise ValueError("%s must have unit stride along its rows" % name)
    _vector_arg("x_scale", x_scale, M, torch.float32)
    _vector_arg("w_scale", w_scale, N, torch.float32)
    if bias is not None:
        _vector_arg("bias", bias, N, dtype)
    if out is not None and (tuple(out.shape) != (M, N) or (N > 1 and out.stride(1) != 1)):
        raise ValueError("out must be %dx%d with unit stride along its rows" % (M, N))
    _need_gpu(X.device, ("X", X), ("W", W), ("x_scale", x_scale), ("w_scale", w_scale), ("bias", bias), ("out", out))

    def call():
        Y = _written(out) if out is not None else torch.empty((M, N), dtype=dtype, device=X.device)
        key = (X.device.index, dtype, M, N, K, X.stride(0), W.stride(0), Y.stride(0), bias is None)
        plan = _plans.get(key)
        if plan is None:
            p = gemm_i8_problem()
            p.M, p.N, p.K = M, N, K
            p.sx, p.sw, p.sy = X.stride(0), W.stride(0), Y.stride(0)
            p.out, p.has_bias = _CODES[dtype], 0 if bias is None else 1
            with _lock:
                plan = _plans.get(key)
                if plan is None:
                    plan = _keep_plan(_plans, key, gemm_i8_plan_create(p, X.device.index))
        gemm_i8_run(plan, X.data_ptr(), x_scale.data_ptr(), W.data_ptr(), w_scale.data_ptr(),
                    bias.data_ptr() if bias is not None else None, Y.data_ptr(), _raw_stream(X.device.index))
        if plain:
            _remember(I8, plan, "gemm_i8_run", 0, (M, N), dtype, out_dtype, X, x_scale, W, w_scale, bias)
        return Y
    return _on_stream(call, X.device, stream, (X, x_scale, W, w_scale, bias, out))
