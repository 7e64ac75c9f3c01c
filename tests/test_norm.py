"""RMS norm and rows in 8 bits: what the entry points refuse, and the gradient
that the GPU tests compare with, against differences (CPU)."""
import ctypes

import pytest
import torch

import dense_tiled_gemm_02_amd as g
from dense_tiled_gemm_02_amd import i8, norm

A = 1 << 20   # a made-up device address, far from the others


def problem(R=4, K=64, **kw):
    p = g.gemm_norm_problem()
    p.R, p.K, p.sx, p.sr, p.sh, p.sy = R, K, K, K, K, K
    p.dtype, p.weight, p.has_residual, p.eps = g.GEMM_BF16, g.GEMM_BF16, 1, 1e-6
    for name, v in kw.items():
        setattr(p, name, v)
    return p


def refused(status, fn):
    with pytest.raises(g.GemmError) as e:
        fn()
    assert e.value.status == status, e.value


def run(p, x=A, r=2 * A, w=3 * A, h=4 * A, y=5 * A, rstd=None):
    norm.gemm_rms_norm(p, x, r, w, h, y, rstd)


INVALID, UNSUPPORTED, WORKSPACE = g.GEMM_ERR_INVALID_ARG, g.GEMM_ERR_UNSUPPORTED, g.GEMM_ERR_WORKSPACE


@pytest.mark.parametrize("status, change", [
    (INVALID, dict(R=-1)), (INVALID, dict(K=-1)), (INVALID, dict(dtype=g.GEMM_I8)), (INVALID, dict(dtype=g.GEMM_F32)),
    (INVALID, dict(dtype=9)), (INVALID, dict(weight=g.GEMM_F16)), (INVALID, dict(weight=g.GEMM_I8)),
    (INVALID, dict(has_residual=2)), (INVALID, dict(eps=0.0)), (INVALID, dict(eps=-1.0)),
    (INVALID, dict(eps=float("nan"))), (INVALID, dict(eps=float("inf"))),
    (UNSUPPORTED, dict(R=(1 << 31) - 1)), (UNSUPPORTED, dict(K=(1 << 31) - 1)),
    (UNSUPPORTED, dict(sx=-64)), (UNSUPPORTED, dict(sr=-64)), (UNSUPPORTED, dict(sh=-64)), (UNSUPPORTED, dict(sy=-1)),
    (INVALID, dict(sy=63)), (INVALID, dict(sh=63)), (INVALID, dict(sx=1 << 61)),
])
def test_refused_problems(status, change):
    refused(status, lambda: run(problem(**change)))
    refused(status, lambda: norm.gemm_rms_norm_i8(problem(**change), A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A))


@pytest.mark.parametrize("status, change", [
    (INVALID, dict(x=None)), (INVALID, dict(r=None)), (INVALID, dict(w=None)), (INVALID, dict(h=None)),
    (INVALID, dict(y=None)), (UNSUPPORTED, dict(x=A + 1)), (UNSUPPORTED, dict(w=A + 1)), (UNSUPPORTED, dict(y=5 * A + 1)),
    (UNSUPPORTED, dict(rstd=6 * A + 2)), (INVALID, dict(y=A)), (INVALID, dict(y=A + 510)), (INVALID, dict(h=2 * A)),
    (INVALID, dict(h=5 * A)), (INVALID, dict(y=3 * A)), (INVALID, dict(rstd=5 * A)),
])
def test_refused_addresses(status, change):
    refused(status, lambda: run(problem(), **change))


def test_residual_only_where_the_problem_has_one():
    refused(INVALID, lambda: run(problem(has_residual=0), h=None))
    refused(INVALID, lambda: run(problem(has_residual=0), r=None))
    refused(INVALID, lambda: norm.gemm_rms_norm_grad(problem(has_residual=0), A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, None))


def test_null_problem():
    assert g.lib().gemm_rms_norm(None, A, A, A, A, A, None, None) == INVALID
    assert g.lib().gemm_rms_norm_i8(None, A, A, A, A, A, A, None) == INVALID
    assert g.lib().gemm_rms_norm_grad(None, A, A, A, A, A, A, A, A, 0, None) == INVALID
    assert g.lib().gemm_rms_norm_grad_workspace(None, ctypes.byref(ctypes.c_size_t())) == INVALID
    assert g.lib().gemm_rms_norm_grad_workspace(ctypes.byref(problem()), None) == INVALID


def test_nothing_to_do_launches_nothing():
    """Without rows, or without values in them, there is no kernel to fail for want of a GPU."""
    run(problem(R=0), None, None, None, None, None)
    run(problem(K=0), None, None, None, None, None)
    norm.gemm_rms_norm_i8(problem(R=0), None, None, None, None, None, None)
    norm.gemm_rms_norm_grad(problem(K=0), None, None, None, None, None, None, None)
    i8.gemm_i8_quantize(None, g.GEMM_F16, 0, 5, 5, None, 5, None)
    refused(INVALID, lambda: norm.gemm_rms_norm_i8(problem(K=0), None, None, None, None, None, None))
    refused(INVALID, lambda: i8.gemm_i8_quantize(None, g.GEMM_F16, 3, 0, 0, None, 0, None))


def test_gradient_needs_its_workspace():
    p = problem()
    need = norm.gemm_rms_norm_grad_workspace(p)
    assert need >= 4 * p.K
    args = (A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A)
    refused(WORKSPACE, lambda: norm.gemm_rms_norm_grad(p, *args))
    refused(WORKSPACE, lambda: norm.gemm_rms_norm_grad(p, *args, 8 * A, need - 1))
    refused(UNSUPPORTED, lambda: norm.gemm_rms_norm_grad(p, *args, 8 * A + 4, need))
    refused(INVALID, lambda: norm.gemm_rms_norm_grad(p, *args, 6 * A, need))
    refused(INVALID, lambda: norm.gemm_rms_norm_grad(p, A, None, *args[2:], 8 * A, need))   # dh goes with the residual
    refused(INVALID, lambda: norm.gemm_rms_norm_grad(problem(sx=63), *args, 8 * A, need))
    assert norm.gemm_rms_norm_grad_workspace(problem(R=0)) == 0


@pytest.mark.parametrize("status, args", [
    (INVALID, (A, 5, 4, 64, 64, 2 * A, 64, 3 * A)), (INVALID, (A, g.GEMM_I8, 4, 64, 64, 2 * A, 64, 3 * A)),
    (INVALID, (A, g.GEMM_F16, -1, 64, 64, 2 * A, 64, 3 * A)), (INVALID, (None, g.GEMM_F16, 4, 64, 64, 2 * A, 64, 3 * A)),
    (INVALID, (A, g.GEMM_F16, 4, 64, 64, None, 64, 3 * A)), (INVALID, (A, g.GEMM_F16, 4, 64, 64, 2 * A, 64, None)),
    (INVALID, (A, g.GEMM_F16, 4, 64, 64, A + 100, 64, 3 * A)), (INVALID, (A, g.GEMM_F16, 4, 64, 64, 2 * A, 60, 3 * A)),
    (UNSUPPORTED, (A + 1, g.GEMM_F16, 4, 64, 64, 2 * A, 64, 3 * A)), (UNSUPPORTED, (A, g.GEMM_F16, 4, 64, 64, 2 * A, 64, 3 * A + 1)),
    (UNSUPPORTED, (A, g.GEMM_F16, 4, 64, -1, 2 * A, 64, 3 * A)),
])
def test_refused_quantizations(status, args):
    refused(status, lambda: i8.gemm_i8_quantize(*args))


def test_torch_calls_refuse_by_name():
    x, w = torch.zeros(3, 8, dtype=torch.bfloat16), torch.ones(8, dtype=torch.bfloat16)
    for call in (norm.rms_norm, norm.rms_norm_i8):
        for error, args in [(TypeError, (x.float(), w)), (ValueError, (x[0], w)), (ValueError, (x.t().contiguous().t(), w)),
                            (TypeError, (x, w.half())), (ValueError, (x, w[:7])), (ValueError, (x, w.expand(2, 8))),
                            (ValueError, (x, torch.ones(1, dtype=torch.bfloat16).expand(8))),
                            (TypeError, (x, w, x.half())), (ValueError, (x, w, x[:2])),
                            (ValueError, (x, w))]:   # the last: no GPU tensors
            with pytest.raises(error):
                call(*args)
    for error, arg in [(TypeError, x.float()), (ValueError, x[0]), (ValueError, x.t()), (ValueError, x)]:
        with pytest.raises(error):
            i8.i8_quantize(arg)


def gradient(dy, dh, h, w, eps):
    """(dx, dw) by the formula, in the tensors' type."""
    K = h.shape[1]
    n = torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    dx = w * dy / n - h * (w * dy * h).sum(1, keepdim=True) / (K * n ** 3)
    return dx if dh is None else dx + dh, (dy * h / n).sum(0)


def test_the_formula_against_differences():
    gen = torch.Generator().manual_seed(3)
    h, dy, dh = (torch.randn(4, 7, generator=gen, dtype=torch.float64) for _ in range(3))
    w = torch.randn(7, generator=gen, dtype=torch.float64)
    eps, step = 0.01, 1e-6
    value = lambda h, w: (dy * h * w / torch.sqrt((h * h).mean(1, keepdim=True) + eps)).sum() + (dh * h).sum()
    dx, dw = gradient(dy, dh, h, w, eps)
    for t, d in ((h, dx), (w, dw)):
        for at in range(t.numel()):
            ends = []
            for s in (step, -step):
                u = t.clone().view(-1)
                u[at] += s
                ends.append(value(u.view_as(t), w) if t is h else value(h, u))
            assert abs((ends[0] - ends[1]) / (2 * step) - d.reshape(-1)[at]) < 1e-8


def test_rows_too_long_for_their_sums_are_refused():
    longest = 1 << 24
    refused(UNSUPPORTED, lambda: norm.gemm_rms_norm(problem(K=longest + 1), A, A, A, A, A, None))
    refused(UNSUPPORTED, lambda: norm.gemm_rms_norm_grad_workspace(problem(K=longest + 1)))
    refused(UNSUPPORTED, lambda: i8.gemm_i8_quantize(A, g.GEMM_BF16, 1, longest + 1, longest + 1, A, longest + 1, A))
    assert norm.gemm_rms_norm_grad_workspace(problem(K=longest)) > 0
