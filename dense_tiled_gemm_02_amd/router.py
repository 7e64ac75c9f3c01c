"""Routing of tokens to experts (include/gemm.h).

    w, ids = route(x @ W, top=2)                                   # softmax over the logits
    w, ids = route(logits, 8, score="sigmoid", bias=b, groups=8, top_groups=4, group_best=2)
    offsets, order = grouped.group_rows(ids.reshape(-1), E)        # to the experts' products

The weights have gradients for the logits.  Argument marshalling only: the work
runs in libgemm.so's HIP kernels.
"""
import ctypes

import torch

from . import (GEMM_BF16, GEMM_F16, GEMM_F32, GEMM_SCORE_SIGMOID, GEMM_SCORE_SOFTMAX, _check, gemm_route_problem, lib)
from .grouped import ROUTE, _need_gpu, _on_stream, _raw_stream, _remembered, _row_operator

_CODES = {torch.float16: GEMM_F16, torch.bfloat16: GEMM_BF16, torch.float32: GEMM_F32}
SCORES = {"softmax": GEMM_SCORE_SOFTMAX, "sigmoid": GEMM_SCORE_SIGMOID}


def gemm_route(problem, logits, bias, weights, ids, stream=None):
    """Device addresses (integers or None) and a hipStream_t (or None)."""
    _check(lib().gemm_route(ctypes.byref(problem), logits, bias, weights, ids, stream))


def gemm_route_grad(problem, logits, ids, dweights, dlogits, stream=None):
    """Device addresses (integers or None) and a hipStream_t (or None)."""
    _check(lib().gemm_route_grad(ctypes.byref(problem), logits, ids, dweights, dlogits, stream))


# ---------------------------------------------------------------- torch convenience

def _logits_arg(logits, score):
    if logits.dtype not in _CODES:
        raise TypeError("logits must be float16, bfloat16 or float32, got %s" % logits.dtype)
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be 2-D with unit stride along the rows, got %s" % (tuple(logits.shape),))
    if score not in SCORES:
        raise ValueError("score must be one of %s, got %r" % (", ".join(SCORES), score))


def route(logits, top, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0,
          stream=None):
    """(weights, ids), float32 and int32, R x top: each row's `top` experts of
    largest score, best first, and scale times their scores, divided by their sum
    with renormalize.

    logits: R x E (up to 1024), float16, bfloat16 or float32; score: "softmax" or
    "sigmoid"; bias: E float32 values added to the scores for the choice alone;
    groups: the experts in that many runs, of which the top_groups strongest take
    part (strength: the sum of a group's best group_best, 1 or 2, scores with
    bias).  Equal scores: the lowest index first.  An expert with a logit or bias
    of -inf or NaN is never chosen; ids that are left over are -1 with weight 0.  A
    row with a NaN logit has NaN weights, and the gradient of the row with -inf there.
    The weights are differentiable for the logits (once, and in reverse mode:
    forward-mode dual logits are refused); in a graph's capture that is refused while
    a graph of the same leaf that was recorded on the default stream is alive.
    Asynchronous on `stream` (default: torch's current stream)."""
    how = (top, SCORES.get(score, -1), groups, top_groups, group_best, 1 if renormalize else 0, float(scale))
    if stream is None:
        pair = _remembered(ROUTE, how, logits, bias)
        if pair is not None:
            return pair
    _logits_arg(logits, score)
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (logits.shape[1],) or
                             (bias.shape[0] > 1 and bias.stride(0) != 1)):
        raise ValueError("bias must be %d contiguous float32 values" % logits.shape[1])
    _need_gpu(logits.device, ("logits", logits), ("bias", bias))
    return _on_stream(lambda: _row_operator("route", ROUTE, stream is None, how, logits, bias), logits.device, stream,
                      (logits, bias))


def route_grad(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0):
    """The gradient of route's weights for the logits (R x E, their type), from
    dweights (R x top float32) and the ids (R x top int32) that route returned."""
    _logits_arg(logits, score)
    if dweights.dtype != torch.float32 or ids.dtype != torch.int32:
        raise TypeError("dweights must be float32 and ids int32, got %s and %s" % (dweights.dtype, ids.dtype))
    if dweights.dim() != 2 or dweights.shape[0] != logits.shape[0] or ids.shape != dweights.shape:
        raise ValueError("dweights and ids must be %d x top, got %s and %s" % (
            logits.shape[0], tuple(dweights.shape), tuple(ids.shape)))
    if not (dweights.is_contiguous() and ids.is_contiguous()):
        raise ValueError("dweights and ids must be contiguous")
    _need_gpu(logits.device, ("logits", logits), ("dweights", dweights), ("ids", ids))

    def call():
        dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        p = gemm_route_problem()
        most = 2 ** 31 - 1   # of the fields; refused
        p.R, p.E, p.top, p.sl = logits.shape[0], min(logits.shape[1], most), min(ids.shape[1], most), logits.stride(0)
        p.groups = p.top_groups = p.group_best = 1
        p.renormalize, p.scale = 1 if renormalize else 0, scale
        p.dtype, p.score = _CODES[logits.dtype], SCORES[score]
        gemm_route_grad(p, logits.data_ptr(), ids.data_ptr(), dweights.data_ptr(), dlogits.data_ptr(),
                        _raw_stream(logits.device.index))
        return dlogits
    return _on_stream(call, logits.device, None, ())
