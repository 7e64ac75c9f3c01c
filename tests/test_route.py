"""Routing: what the entry points refuse, and the oracle of the GPU tests: its
choice on small rows by hand, its gradient against differences (CPU)."""
import math

import pytest
import torch

import dense_tiled_gemm_02_amd as g
from dense_tiled_gemm_02_amd import router

A = 1 << 20


def problem(**kw):
    p = g.gemm_route_problem()
    p.R, p.sl, p.E, p.top = 4, 16, 16, 2
    p.groups, p.top_groups, p.group_best = 4, 2, 2
    p.has_bias, p.renormalize, p.scale, p.dtype, p.score = 1, 1, 1.0, g.GEMM_BF16, g.GEMM_SCORE_SIGMOID
    for name, v in kw.items():
        setattr(p, name, v)
    return p


def refused(status, fn):
    with pytest.raises(g.GemmError) as e:
        fn()
    assert e.value.status == status, e.value


INVALID, UNSUPPORTED = g.GEMM_ERR_INVALID_ARG, g.GEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("status, change", [
    (INVALID, dict(R=-1)), (INVALID, dict(E=0)), (INVALID, dict(E=-4)), (INVALID, dict(top=0)), (INVALID, dict(top=9)),
    (INVALID, dict(dtype=g.GEMM_I8)), (INVALID, dict(dtype=7)), (INVALID, dict(score=2)), (INVALID, dict(has_bias=2)),
    (INVALID, dict(renormalize=-1)), (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=float("inf"))),
    (INVALID, dict(groups=0)), (INVALID, dict(groups=3)), (INVALID, dict(top_groups=0)), (INVALID, dict(top_groups=5)),
    (INVALID, dict(group_best=0)), (INVALID, dict(group_best=3)), (UNSUPPORTED, dict(E=1028, sl=1028)),
    (UNSUPPORTED, dict(E=1024, sl=1024, top=65)), (UNSUPPORTED, dict(E=130, groups=65, top_groups=1)),
    (UNSUPPORTED, dict(R=(1 << 31) - 1)), (UNSUPPORTED, dict(sl=-1)), (INVALID, dict(sl=1 << 59)),
])
def test_refused_problems(status, change):
    refused(status, lambda: router.gemm_route(problem(**change), A, 2 * A, 3 * A, 4 * A))
    refused(status, lambda: router.gemm_route_grad(problem(**change), A, 2 * A, 3 * A, 4 * A))


@pytest.mark.parametrize("status, args", [
    (INVALID, (None, 2 * A, 3 * A, 4 * A)), (INVALID, (A, None, 3 * A, 4 * A)), (INVALID, (A, 2 * A, None, 4 * A)),
    (INVALID, (A, 2 * A, 3 * A, None)), (UNSUPPORTED, (A + 1, 2 * A, 3 * A, 4 * A)), (UNSUPPORTED, (A, 2 * A + 2, 3 * A, 4 * A)),
    (UNSUPPORTED, (A, 2 * A, 3 * A + 1, 4 * A)), (UNSUPPORTED, (A, 2 * A, 3 * A, 4 * A + 2)), (INVALID, (A, 2 * A, A, 4 * A)),
    (INVALID, (A, 2 * A, 3 * A, 3 * A + 16)), (INVALID, (A, 2 * A, 2 * A, 4 * A)),
])
def test_refused_addresses(status, args):
    refused(status, lambda: router.gemm_route(problem(), *args))


def test_more_refusals():
    refused(INVALID, lambda: router.gemm_route(problem(has_bias=0), A, 2 * A, 3 * A, 4 * A))
    refused(INVALID, lambda: router.gemm_route_grad(problem(), A, 2 * A, 3 * A, None))
    refused(INVALID, lambda: router.gemm_route_grad(problem(), A, 2 * A, 3 * A, 3 * A))
    assert g.lib().gemm_route(None, A, A, A, A, None) == INVALID
    assert g.lib().gemm_route_grad(None, A, A, A, A, None) == INVALID
    router.gemm_route(problem(R=0), None, None, None, None)
    router.gemm_route_grad(problem(R=0), None, None, None, None)


def test_torch_calls_refuse_by_name():
    l = torch.zeros(3, 8)
    for error, args, kw in [(TypeError, (l.double(), 2), {}), (ValueError, (l[0], 2), {}), (ValueError, (l.t(), 2), {}),
                            (ValueError, (l, 2), dict(score="top")), (ValueError, (l, 2), dict(bias=torch.zeros(7))),
                            (ValueError, (l, 2), dict(bias=torch.zeros(8).half())), (ValueError, (l, 2), {})]:
        with pytest.raises(error):
            router.route(*args, **kw)
    w, ids = torch.zeros(3, 2), torch.zeros(3, 2, dtype=torch.int32)
    for error, args in [(TypeError, (w.half(), l, ids)), (TypeError, (w, l, ids.long())), (ValueError, (w[:2], l, ids)),
                        (ValueError, (w, l, ids[:, :1])), (ValueError, (w.t().contiguous().t(), l, ids)), (ValueError, (w, l, ids))]:
        with pytest.raises(error):
            router.route_grad(*args)


# ---------------------------------------------------------------- the oracle

def scores(l, score):
    """64-bit scores; NaN logits have none, infinite ones share the whole."""
    l = torch.where(torch.isnan(l), -math.inf, l.double())
    if score == "sigmoid":
        return torch.sigmoid(l)
    top = l.max(1, keepdim=True).values
    e = torch.where(l == top, 1.0, torch.exp(l - torch.where(torch.isinf(top), 0.0, top)))
    e = torch.where((top == math.inf) & (l < top), 0.0, e)
    return e / e.sum(1, keepdim=True)


def oracle(l, top, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0):
    """(weights, ids) of CPU logits, row by row in 64 bits."""
    R, E = l.shape
    p = scores(l, score)
    had = ~torch.isnan(l) & (l != -math.inf)
    if bias is not None:
        had &= ~torch.isnan(bias) & (bias != -math.inf)
    weights, ids = torch.zeros(R, top, dtype=torch.float64), torch.full((R, top), -1, dtype=torch.int32)
    c = p if bias is None else p + bias.double()
    order = l.double() if bias is None else c   # without a bias, scores that 64 bits cannot tell apart go by the logits
    orders, summands, havings = order.tolist(), c.tolist(), had.tolist()
    for r in range(R):
        rank, of_group, having = orders[r], summands[r], havings[r]
        left = [e for e in range(E) if having[e]]
        if groups > 1:
            per = E // groups
            strength = []
            for k in range(groups):
                mine = [e for e in left if e // per == k]
                by = rank if group_best == 1 else of_group
                best = sorted((by[e] for e in mine), reverse=True)[:group_best]
                if best:
                    strength.append((-sum(best), k))
            kept = {k for _, k in sorted(strength)[:top_groups]}
            left = [e for e in left if e // per in kept]
        chosen = sorted(left, key=lambda e: (-rank[e], e))[:top]
        if not chosen:
            continue
        ids[r, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
        w = p[r, chosen]
        if renormalize:
            if score == "softmax":
                w = scores(l[r:r + 1, chosen], "softmax")[0]
            elif float(w.sum()) < 1e-290:   # shares of what 64 bits cannot hold: e^l / (1 + e^l) is e^l
                w = torch.softmax(l[r, chosen].double(), 0)
            else:
                w = w / w.sum()
        weights[r, :len(chosen)] = w * scale if not torch.isnan(l[r]).any() else math.nan
    return weights, ids


def oracle_grad(dw, l, ids, score, renormalize, scale):
    """dlogits in 64 bits."""
    p = scores(l, score)
    real = ids >= 0
    at = ids.long().clamp(min=0)
    g = dw.double() * scale * real
    if renormalize:
        u = (scores(torch.where(real, l.double().gather(1, at), -math.inf), "softmax") if score == "softmax"
             else p.gather(1, at) * real / (p.gather(1, at) * real).sum(1, keepdim=True))
        u = torch.where(real, u, 0.0)
        d = u * (g - (g * u).sum(1, keepdim=True))
        if score == "sigmoid":
            d = d * torch.sigmoid(-l.double().gather(1, at))
        return torch.zeros_like(p).scatter_add_(1, at, d * real)
    if score == "sigmoid":
        s = p.gather(1, at)
        return torch.zeros_like(p).scatter_add_(1, at, g * s * (1 - s))
    full = torch.zeros_like(p).scatter_add_(1, at, g)
    return p * (full - (full * p).sum(1, keepdim=True))


def test_oracle_by_hand():
    l = torch.tensor([[0.0, 3.0, 3.0, -1.0]])
    assert oracle(l, 3)[1].tolist() == [[1, 2, 0]]
    assert oracle(l, 1, bias=torch.tensor([2.0, 0.0, 0.0, 0.0]))[1].tolist() == [[0]]
    w, ids = oracle(l, 2, score="sigmoid", renormalize=False, scale=2.0)
    assert ids.tolist() == [[1, 2]] and abs(float(w[0, 0]) - 2 / (1 + math.exp(-3.0))) < 1e-15
    # groups {0, 1} and {2, 3}: the first has the larger pair, the second the larger best after a bias
    l = torch.tensor([[2.0, 1.9, 2.5, -4.0]])
    assert oracle(l, 2, score="sigmoid", groups=2, group_best=2)[1].tolist() == [[0, 1]]
    assert oracle(l, 2, score="sigmoid", groups=2, group_best=1)[1].tolist() == [[2, 3]]
    w, ids = oracle(torch.tensor([[-math.inf, 1.0, -math.inf]]), 2)
    assert ids.tolist() == [[1, -1]] and w.tolist() == [[1.0, 0.0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_oracle_gradient_against_differences(score, renormalize):
    gen = torch.Generator().manual_seed(1)
    l = torch.randn(5, 9, generator=gen, dtype=torch.float64)
    dw = torch.randn(5, 3, generator=gen, dtype=torch.float64)
    _, ids = oracle(l, 3, score=score)
    value = lambda l: (oracle(l, 3, score=score, renormalize=renormalize, scale=1.7)[0] * dw).sum()
    d = oracle_grad(dw, l, ids, score, renormalize, 1.7)
    for r in range(5):
        for e in range(9):
            ends = []
            for s in (1e-6, -1e-6):
                m = l.clone()
                m[r, e] += s
                ends.append(value(m))
            assert abs((ends[0] - ends[1]) / 2e-6 - d[r, e]) < 1e-8
