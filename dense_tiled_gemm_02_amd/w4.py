"""Matrix-vector products with 4-bit weights and group scales (include/gemm.h).

    q, scale, zero = w4_quantize(W, group=128)             # W: N x K or E x N x K
    Y = w4_matvec(X, q, scale, zero, group=128)            # Y = X W^T for a few rows of X
    Y = w4_matvec(X, q, scale, experts=ids, group=128)     # row m through expert ids[m]

Argument marshalling only: the product runs in libgemm.so's HIP kernels.
"""
import ctypes
import threading

import torch

from . import GEMM_BF16, GEMM_F16, _check, _keep_plan, _p, gemm_w4_problem, lib
from .grouped import W4, _need_gpu, _on_stream, _raw_stream, _remember, _remembered

_CODES = {torch.float16: GEMM_F16, torch.bfloat16: GEMM_BF16}


class W4Plan:
    """Owns one gemm_w4_plan*; destroyed with the object."""

    def __init__(self, handle, problem):
        self.handle = handle
        self.problem = problem

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            lib().gemm_w4_plan_destroy(h)

    def describe(self):
        buf = ctypes.create_string_buffer(1024)
        _check(lib().gemm_w4_plan_describe(self.handle, buf, len(buf)))
        return buf.value.decode()


def gemm_w4_plan_create(problem, device=0):
    h = _p()
    _check(lib().gemm_w4_plan_create(ctypes.byref(problem), device, ctypes.byref(h)))
    return W4Plan(h, problem)


def gemm_w4_plan_create_for(problem, info):
    h = _p()
    _check(lib().gemm_w4_plan_create_for(ctypes.byref(problem), ctypes.byref(info), ctypes.byref(h)))
    return W4Plan(h, problem)


def gemm_w4_run(plan, X, W, S, Z, expert_ids, Y, stream=None):
    """Device addresses (integers or None) and a hipStream_t (or None)."""
    _check(lib().gemm_w4_run(plan.handle, X, W, S, Z, expert_ids, Y, stream))


# ---------------------------------------------------------------- torch convenience

_plans = {}
_lock = threading.Lock()   # guards _plans


def w4_matvec(X, W, scale, zeros=None, group=128, experts=None, out=None, stream=None):
    """Y[m, n] = sum_k X[m, k] (q[n, k] - zero[n, k // group]) scale[n, k // group].

    X: M x K, float16 or bfloat16.  W: N x K/2 uint8, two k per byte, even k in
    the low nibble; scale: N x ceil(K / group) of X's dtype; zeros: the same
    shape, uint8 (None: 8).  experts: one id per row of X (int32 or int64), W,
    scale and zeros then with a leading dimension of experts; a row whose id is
    outside it gives zeros.  group: 32, 64 or 128.  Asynchronous on `stream`
    (default: torch's current stream)."""
    plain = out is None and stream is None
    if plain:
        Y = _remembered(W4, group, X, W, scale, zeros, experts)
        if Y is not None:
            return Y
    if X.dtype not in _CODES:
        raise TypeError("X must be float16 or bfloat16, got %s" % X.dtype)
    if W.dtype != torch.uint8 or (zeros is not None and zeros.dtype != torch.uint8):
        raise TypeError("W and zeros must be uint8")
    if scale.dtype != X.dtype:
        raise TypeError("scale has dtype %s, expected %s" % (scale.dtype, X.dtype))
    nd = 2 if experts is None else 3
    if X.dim() != 2 or W.dim() != nd:
        raise ValueError("X must be 2-D and W %d-D, got %s and %s" % (nd, tuple(X.shape), tuple(W.shape)))
    if group <= 0:
        raise ValueError("group must be positive, got %d" % group)
    M, K = X.shape
    N = W.shape[-2]
    if K != 2 * W.shape[-1]:
        raise ValueError("X has %d columns, W %d" % (K, 2 * W.shape[-1]))
    groups = W.shape[:-1] + (-(-K // group),)
    if scale.shape != groups or (zeros is not None and zeros.shape != groups):
        raise ValueError("scale and zeros must be %s" % (tuple(groups),))
    for name, t in (("X", X), ("W", W), ("scale", scale), ("zeros", zeros)):
        if t is not None and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError("%s must have unit stride along its rows" % name)
    if experts is not None:
        if experts.dtype not in (torch.int32, torch.int64):
            raise TypeError("experts must be int32 or int64, got %s" % experts.dtype)
        if tuple(experts.shape) != (M,) or (M > 1 and experts.stride(0) != 1):
            raise ValueError("experts must be %d contiguous ids" % M)
    if out is not None and (out.dtype != X.dtype or tuple(out.shape) != (M, N) or (N > 1 and out.stride(1) != 1)):
        raise ValueError("out must be %s of %dx%d with unit stride along its rows" % (X.dtype, M, N))
    _need_gpu(X.device, ("X", X), ("W", W), ("scale", scale), ("zeros", zeros), ("experts", experts), ("out", out))

    def call():
        Y = out if out is not None else torch.empty((M, N), dtype=X.dtype, device=X.device)
        if experts is not None and W.shape[0] == 0:   # no matrix: every row is outside
            return Y.zero_()
        key = (X.device.index, X.dtype, M, X.stride(0), W.shape, W.stride(), scale.stride(),
               None if zeros is None else zeros.stride(), group, None if experts is None else experts.dtype,
               Y.stride(0))
        plan = _plans.get(key)
        if plan is None:
            p = gemm_w4_problem()
            p.M, p.N, p.K, p.group = M, N, K, group
            p.sx = X.stride(0) if M > 1 and K > 0 else 0   # strides that no access uses are not looked at
            p.sy = Y.stride(0)
            p.sw_n, p.ss_n = W.stride(-2) if N > 1 and K > 0 else 0, scale.stride(-2)
            if experts is not None:
                p.experts, p.id_bytes = W.shape[0], experts.element_size()
                p.sw_e, p.ss_e = W.stride(0) if W.shape[0] > 1 and K > 0 else 0, scale.stride(0)
            if zeros is not None:
                p.has_zeros, p.sz_n = 1, zeros.stride(-2)
                p.sz_e = zeros.stride(0) if experts is not None else 0
            p.dtype = _CODES[X.dtype]
            with _lock:
                plan = _plans.get(key)
                if plan is None:
                    plan = _keep_plan(_plans, key, gemm_w4_plan_create(p, X.device.index))
        gemm_w4_run(plan, X.data_ptr(), W.data_ptr(), scale.data_ptr(),
                    zeros.data_ptr() if zeros is not None else None,
                    experts.data_ptr() if experts is not None else None, Y.data_ptr(),
                    _raw_stream(X.device.index))
        if plain:
            _remember(W4, plan, "gemm_w4_run", 0, (M, N), X.dtype, group, X, W, scale, zeros, experts)
        return Y
    return _on_stream(call, X.device, stream, (X, W, scale, zeros, experts, out))


def w4_quantize(W, group=128, zeros=False):
    """(q, scale, zero) of w4_matvec for W (N x K or E x N x K, float16 or
    bfloat16; K a multiple of 32): round-to-nearest against each group's
    largest magnitude (zero is None), or, with zeros, against its range."""
    if W.dtype not in _CODES:
        raise TypeError("W must be float16 or bfloat16, got %s" % W.dtype)
    if W.dim() == 0:
        raise ValueError("W must have rows")
    if group <= 0:
        raise ValueError("group must be positive, got %d" % group)
    K = W.shape[-1]
    if K % 32:
        raise ValueError("K=%d must be a multiple of 32" % K)
    n = -(-K // group)
    w = torch.nn.functional.pad(W.float(), (0, n * group - K)).unflatten(-1, (n, group))
    tiny = torch.finfo(W.dtype).tiny * torch.finfo(W.dtype).eps   # the smallest scale above zero
    if zeros:
        lo, hi = w.amin(-1).clamp(max=0.0), w.amax(-1).clamp(min=0.0)
        scale = ((hi - lo) / 15).clamp(min=tiny).to(W.dtype)
        zero = torch.round(-lo / scale.float()).clamp(0, 15)
    else:
        scale = (w.abs().amax(-1) / 7).clamp(min=tiny).to(W.dtype)
        zero = torch.full_like(scale, 8.0, dtype=torch.float32)
    q = torch.round(w / scale.float()[..., None] + zero[..., None]).clamp(0, 15).to(torch.uint8)
    q = q.flatten(-2)[..., :K]
    packed = q[..., 0::2] | (q[..., 1::2] << 4)
    return packed.contiguous(), scale, zero.to(torch.uint8) if zeros else None
