"""Products grouped by expert with ragged sizes (include/gemm.h).

The rows of an operand are sorted by group, and a device table of offsets
(groups + 1, int32) says which rows each group owns; the host never reads it,
so nothing here synchronizes and every call can be captured in a graph.

    offsets, order = group_rows(ids, E)              # the router's ids -> table and row order
    D = grouped_matmul(X[order], W, offsets)         # W: E x K x N, or the transposed view of E x N x K
    dX = grouped_matmul(dD, W.transpose(1, 2), offsets)
    dW = grouped_wgrad(X[order], dD, offsets)

`grouped_linear` is grouped_matmul with these gradients, for autograd (of any order).
Argument marshalling only: the work runs in libgemm.so's HIP kernels.
"""
import contextlib
import ctypes
import threading

import torch

from . import (GEMM_BF16, GEMM_F16, GEMM_GROUPED_OUT_F32, GEMM_GROUPED_OUT_SAME, GEMM_GROUPED_REDUCE,
               GEMM_GROUPED_ROWS, _check, _force, _i32, _i64, _keep_plan, _p, binding, gemm_config,
               gemm_grouped_problem, lib)

_CODES = {torch.float16: GEMM_F16, torch.bfloat16: GEMM_BF16}


class GroupedPlan:
    """Owns one gemm_grouped_plan*; destroyed with the object."""

    def __init__(self, handle, problem):
        self.handle = handle
        self.problem = problem
        self.workspace = gemm_grouped_workspace(self)

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            lib().gemm_grouped_plan_destroy(h)

    @property
    def config(self):
        c = gemm_config()
        _check(lib().gemm_grouped_plan_config(self.handle, ctypes.byref(c)))
        return c

    def launch(self):
        g, t, l = _i64(), _i32(), _i64()
        _check(lib().gemm_grouped_plan_launch(self.handle, ctypes.byref(g), ctypes.byref(t), ctypes.byref(l)))
        return g.value, t.value, l.value

    def describe(self):
        buf = ctypes.create_string_buffer(1024)
        _check(lib().gemm_grouped_plan_describe(self.handle, buf, len(buf)))
        return buf.value.decode()


def gemm_grouped_plan_create(problem, device=0, force=None):
    h = _p()
    _check(lib().gemm_grouped_plan_create(ctypes.byref(problem), device, _force(force), ctypes.byref(h)))
    return GroupedPlan(h, problem)


def gemm_grouped_plan_create_for(problem, info, force=None):
    h = _p()
    _check(lib().gemm_grouped_plan_create_for(ctypes.byref(problem), ctypes.byref(info), _force(force),
                                              ctypes.byref(h)))
    return GroupedPlan(h, problem)


def gemm_grouped_run(plan, A, B, offsets, D, stream=None):
    """Device addresses (integers or None) and a hipStream_t (or None)."""
    _check(lib().gemm_grouped_run(plan.handle, A, B, offsets, D, stream))


def gemm_grouped_workspace(plan):
    n = ctypes.c_size_t()
    _check(lib().gemm_grouped_workspace(plan.handle, ctypes.byref(n)))
    return n.value


def gemm_grouped_run_parts(plan, A, B, offsets, D, workspace, workspace_bytes, stream=None):
    """gemm_grouped_run with a workspace (an address, or None) for the parts of long groups."""
    _check(lib().gemm_grouped_run_parts(plan.handle, A, B, offsets, D, workspace, workspace_bytes, stream))


def gemm_group_rows_workspace(R, groups):
    n = ctypes.c_size_t()
    _check(lib().gemm_group_rows_workspace(R, groups, ctypes.byref(n)))
    return n.value


def gemm_group_rows(ids, id_bytes, R, groups, offsets, order, workspace=None, workspace_bytes=0, stream=None):
    """Device addresses (integers or None) and a hipStream_t (or None)."""
    _check(lib().gemm_group_rows(ids, id_bytes, R, groups, offsets, order, workspace, workspace_bytes, stream))


# ---------------------------------------------------------------- torch convenience

_plans = {}
_lock = threading.Lock()   # guards _plans

# The plain calls (no out, config or stream) that passed every check are
# remembered by _binding.so, by what the checks look at: the operands' types,
# shapes, strides and devices.  A call found there goes straight to the launch:
# 4.1 to 4.9 us of host time instead of 7.4, which is what the smallest products take.
MATMUL, WGRAD, ROWS, W4, NORM, NORM_I8, I8_ROWS, I8, ROUTE = range(9)   # csrc/binding.cpp
_call = None
_raw_stream = torch._C._cuda_getCurrentRawStream


def _address(name):
    return ctypes.cast(getattr(lib(), name), ctypes.c_void_p).value


def _remembered(kind, extra, *tensors):
    """The call's outputs, or None where it has to be checked first."""
    global _call
    if _call is None:
        _call = _native().call
    r = _call(kind, extra, *tensors)
    if type(r) is int:
        _check(r)
    return r


_bound = None


def _native():
    """_binding.so, which knows where libgemm.so's row operators are."""
    global _bound
    if _bound is None:
        b = binding()
        b.functions(*[_address(name) for name in (
            "gemm_rms_norm", "gemm_rms_norm_i8", "gemm_rms_norm_grad_workspace", "gemm_rms_norm_grad", "gemm_i8_quantize",
            "gemm_route", "gemm_route_grad", "gemm_last_error")])
        _bound = b
    return _bound


def _row_operator(name, kind, remember, extra, *tensors):
    """A row operator of _binding.so on checked arguments; `remember`: such calls go there at once from now on."""
    r = getattr(_native(), name)(*tensors, *(() if extra is None else (extra,)))
    if type(r) is int:
        _check(r)
    if remember:
        binding().remember(kind, None, 0, 0, 0, (), torch.uint8, extra, tensors)
    return r


def _remember(kind, plan, run, workspace, sizes, dtype, extra, *tensors):
    binding().remember(kind, plan, plan.handle.value if plan is not None else 0, _address(run), workspace, sizes,
                       dtype, extra, tensors)


def _need_gpu(device, *named):
    """Every tensor on `device`, a GPU."""
    for name, t in named:
        if t is not None and (not t.is_cuda or t.device != device):
            raise ValueError("%s must be on %s, a GPU" % (name, device) if device.type == "cuda"
                             else "%s must be a GPU tensor" % name)


@contextlib.contextmanager
def _another_stream(device, stream, inputs):
    """The caller's stream as torch's current one: outputs and workspaces made
    inside belong to it, and the allocator is told that it reads the inputs."""
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(s):
        for t in inputs:
            if t is not None:
                t.record_stream(s)
        yield


def _on_stream(fn, device, stream, inputs):
    """fn() with `stream` (torch stream, hipStream_t or None: torch's current
    one) and the tensors' device current.  A caller's `out` counts as an input."""
    if stream is None and device.index == torch.cuda.current_device():
        return fn()
    with torch.cuda.device(device):
        if stream is None:
            return fn()
        with _another_stream(device, stream, inputs):
            return fn()


def _written(out):
    """The caller's `out`, noted as modified: autograd then finds a value that it
    holds for a backward pass overwritten."""
    torch.autograd.graph.increment_version(out)
    return out


def _offsets_arg(offsets, groups, device):
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.shape[0] != groups + 1:
        raise ValueError("offsets must be %d int32 values, got %s %s" % (groups + 1, offsets.dtype,
                                                                        tuple(offsets.shape)))
    if offsets.stride(0) != 1 and groups > 0:
        raise ValueError("offsets must be contiguous")


def _launch(plan, A, B, offsets, out, stream):
    if plan.workspace:   # released on return: later work of this stream may reuse it, in order
        ws = A.new_empty(plan.workspace, dtype=torch.uint8)
        gemm_grouped_run_parts(plan, A.data_ptr(), B.data_ptr(), offsets.data_ptr(), out.data_ptr(), ws.data_ptr(),
                               plan.workspace, stream)
    else:
        gemm_grouped_run(plan, A.data_ptr(), B.data_ptr(), offsets.data_ptr(), out.data_ptr(), stream)


def _run(kind, A, B, offsets, out, groups, P, Q, accumulate, config):
    sa, sb, sd = A.stride(), B.stride(), out.stride()
    key = (A.device.index, kind, A.dtype, out.dtype, accumulate, groups, A.shape[0], P, Q, sa, sb, sd,
           tuple(sorted(config.items())) if config else None)
    plan = _plans.get(key)
    if plan is None:
        p = gemm_grouped_problem()
        p.groups, p.R, p.P, p.Q = groups, A.shape[0], P, Q
        p.sa_r, p.sa_p = sa
        if kind == GEMM_GROUPED_ROWS:
            p.sb_g, p.sb_r, p.sb_q = sb
            p.sd_r = sd[0]
        else:
            p.sb_r, p.sb_q = sb
            p.sd_g, p.sd_r = sd[0], sd[1]
        if Q > 1 and sd[-1] != 1:
            raise ValueError("out must have unit stride along its last dimension")
        p.dtype, p.kind = _CODES[A.dtype], kind
        p.out = GEMM_GROUPED_OUT_F32 if out.dtype == torch.float32 else GEMM_GROUPED_OUT_SAME
        p.accumulate = 1 if accumulate else 0
        with _lock:
            plan = _plans.get(key)
            if plan is None:
                plan = _keep_plan(_plans, key, gemm_grouped_plan_create(p, A.device.index, config))
    _launch(plan, A, B, offsets, out, _raw_stream(A.device.index))
    return plan


def _operands(A, B, nb):
    if A.dtype not in _CODES:
        raise TypeError("only float16 and bfloat16 operands are supported, got %s" % A.dtype)
    if B.dtype != A.dtype:
        raise TypeError("operands have dtypes %s and %s" % (A.dtype, B.dtype))
    if A.dim() != 2 or B.dim() != nb:
        raise ValueError("operands must be 2-D and %d-D, got %s and %s" % (nb, tuple(A.shape), tuple(B.shape)))


def grouped_matmul(A, B, offsets, out=None, config=None, stream=None):
    """D[i] = A[i] x B[g] for offsets[g] <= i < offsets[g + 1]; rows of no group
    are zeros.  A: R x K, B: E x K x N (any strides: the transposed view of an
    E x N x K weight, or of the forward's weight for the input gradient),
    float16 or bfloat16; offsets: E + 1 int32 on the GPU, not decreasing.
    config: optional dict of gemm_config fields to force.  Asynchronous on
    `stream` (default: torch's current stream)."""
    plain = out is None and config is None and stream is None
    if plain:
        D = _remembered(MATMUL, None, A, B, offsets)
        if D is not None:
            return D
    _operands(A, B, 3)
    E, K, N = B.shape
    R = A.shape[0]
    if A.shape[1] != K:
        raise ValueError("inner dimensions differ: %s x %s" % (tuple(A.shape), tuple(B.shape)))
    _need_gpu(A.device, ("A", A), ("B", B), ("offsets", offsets), ("out", out))
    _offsets_arg(offsets, E, A.device)
    if out is not None and (out.dtype != A.dtype or tuple(out.shape) != (R, N)):
        raise ValueError("out must be %s of %dx%d" % (A.dtype, R, N))

    def call():
        D = _written(out) if out is not None else torch.empty((R, N), dtype=A.dtype, device=A.device)
        plan = _run(GEMM_GROUPED_ROWS, A, B, offsets, D, E, K, N, False, config)
        if plain:
            _remember(MATMUL, plan, "gemm_grouped_run_parts", plan.workspace, (R, N), A.dtype, None, A, B, offsets)
        return D
    return _on_stream(call, A.device, stream, (A, B, offsets, out))


def grouped_wgrad(A, G, offsets, out=None, out_dtype=None, accumulate=False, config=None, stream=None):
    """D[e] = A_e^T x G_e (K x N) over each group's rows: the gradient of the
    weights of grouped_matmul.  A: R x K, G: R x N; the gradient of a weight
    stored N x K is grouped_wgrad(G, A).  out_dtype: the operands' dtype (the
    default) or float32.  An empty group gives zeros.  accumulate: add to `out`
    (E x K x N) instead of overwriting it."""
    plain = out is None and config is None and stream is None and not accumulate
    if plain:
        D = _remembered(WGRAD, out_dtype, A, G, offsets)
        if D is not None:
            return D
    _operands(A, G, 2)
    if A.shape[0] != G.shape[0]:
        raise ValueError("row counts differ: %s and %s" % (tuple(A.shape), tuple(G.shape)))
    if offsets.dim() != 1 or offsets.shape[0] == 0:
        raise ValueError("offsets must hold at least one value in one dimension")
    E, K, N = offsets.shape[0] - 1, A.shape[1], G.shape[1]
    _need_gpu(A.device, ("A", A), ("G", G), ("offsets", offsets), ("out", out))
    _offsets_arg(offsets, E, A.device)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    dtype = out.dtype if out is not None else (out_dtype or A.dtype)
    if dtype not in (A.dtype, torch.float32) or (out_dtype is not None and dtype != out_dtype):
        raise TypeError("the gradient is %s or float32, got %s" % (A.dtype, out_dtype or dtype))
    if out is not None and tuple(out.shape) != (E, K, N):
        raise ValueError("out must be %dx%dx%d" % (E, K, N))

    def call():
        D = _written(out) if out is not None else torch.empty((E, K, N), dtype=dtype, device=A.device)
        plan = _run(GEMM_GROUPED_REDUCE, A, G, offsets, D, E, K, N, accumulate, config)
        if plain:
            _remember(WGRAD, plan, "gemm_grouped_run_parts", plan.workspace, (E, K, N), dtype, out_dtype, A, G, offsets)
        return D
    return _on_stream(call, A.device, stream, (A, G, offsets, out))


def group_rows(ids, groups, stream=None):
    """(offsets, order), both int32, for one group id per row (int32 or int64):
    order lists the rows by ascending id, rows of one id in their own order and
    rows whose id is outside [0, groups) last; offsets (groups + 1) holds each
    group's first place in it."""
    if stream is None:
        pair = _remembered(ROWS, groups, ids)
        if pair is not None:
            return pair
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be int32 or int64, got %s" % ids.dtype)
    if ids.dim() != 1 or (ids.shape[0] > 1 and ids.stride(0) != 1):
        raise ValueError("ids must be one contiguous dimension")
    _need_gpu(ids.device, ("ids", ids))

    R = ids.shape[0]

    def call():
        need = gemm_group_rows_workspace(R, groups)
        offsets = torch.empty(groups + 1, dtype=torch.int32, device=ids.device)
        order = torch.empty(R, dtype=torch.int32, device=ids.device)
        ws = torch.empty(need, dtype=torch.uint8, device=ids.device) if need else None
        gemm_group_rows(ids.data_ptr(), ids.element_size(), R, groups, offsets.data_ptr(), order.data_ptr(),
                        ws.data_ptr() if need else None, need, _raw_stream(ids.device.index))
        if stream is None:
            _remember(ROWS, None, "gemm_group_rows", need, (groups, R, ids.element_size()), torch.int32, groups, ids)
        return offsets, order
    return _on_stream(call, ids.device, stream, (ids,))


# Each one's gradients are made of the other, so they have derivatives of any
# order.  A backward pass that no one differentiates calls the operators directly.
def _differentiable():
    return (grouped_linear, _GroupedWgrad.apply) if torch.is_grad_enabled() else (grouped_matmul, grouped_wgrad)


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, offsets):
        ctx.save_for_backward(x, weight, offsets)
        return grouped_matmul(x, weight, offsets)

    @staticmethod
    def backward(ctx, grad):
        x, weight, offsets = ctx.saved_tensors
        matmul, wgrad = _differentiable()
        grad = grad.contiguous()   # an expanded gradient (of a sum) would take the element-wise tiles
        dx = matmul(grad, weight.transpose(1, 2), offsets) if ctx.needs_input_grad[0] else None
        dw = wgrad(x, grad, offsets) if ctx.needs_input_grad[1] else None
        return dx, dw, None


class _GroupedWgrad(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, grad, offsets):
        ctx.save_for_backward(x, grad, offsets)
        return grouped_wgrad(x, grad, offsets)

    @staticmethod
    def backward(ctx, d):
        x, grad, offsets = ctx.saved_tensors
        matmul, _ = _differentiable()
        d = d.contiguous()
        dx = matmul(grad, d.transpose(1, 2), offsets) if ctx.needs_input_grad[0] else None
        dgrad = matmul(x, d, offsets) if ctx.needs_input_grad[1] else None
        return dx, dgrad, None


def grouped_linear(x, weight, offsets):
    """grouped_matmul(x, weight, offsets) with gradients, of any order, for x
    (R x K) and weight (E x K x N)."""
    return _GroupedLinear.apply(x, weight, offsets)
