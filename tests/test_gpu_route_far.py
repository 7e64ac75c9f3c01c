"""Routing by biased and grouped scores of logits far from zero, where e^-l passes
fp32's range or the score does: the choice is the one of 64-bit scores (GPU).

A weight is scale s / sum, with s the score, or, renormalized, e^(l - the largest
chosen l) or a like share.  fp32's exponential of less than 2^-126 is 0, which is
all of s; the sum is 1 or holds the largest share, at least 1/2 (a sigmoid of
l >= 0, or 1 / (1 + e^l) of l < 0): the weight is then off by 2 scale 2^-126 at
most.  Else it is off as in test_gpu_route.py: 2^-18 of itself and 2^-23 for every
unit between the logits."""
import math

import pytest
import torch

from dense_tiled_gemm_02_amd import router
from test_gpu_route import TYPES
from test_route import oracle

pytestmark = pytest.mark.gpu

E = 64


def check(l, top, scale=1.0, **kw):
    w, ids = router.route(l.cuda(), top, scale=scale, **{k: v.cuda() if torch.is_tensor(v) else v for k, v in kw.items()})
    want, want_ids = oracle(l, top, scale=scale, **kw)
    assert torch.equal(ids.cpu(), want_ids)
    assert bool((want_ids >= 0).all())   # none of these inputs leaves a row short of experts
    apart = 420.0   # logits are within 210 of zero
    assert bool(((w.cpu().double() - want).abs() <= want * (2.0 ** -18 + apart * 2.0 ** -23) + 2 * scale * 2.0 ** -126).all())


def sweep(lo, hi):
    """Rows that hold every quarter of [lo, hi] in a random order."""
    gen = torch.Generator().manual_seed(int(hi))
    l = torch.arange(lo, hi, 0.25)
    l = torch.cat([l[torch.randperm(l.numel(), generator=gen)] for _ in range(3)])
    return l[:l.numel() // E * E].reshape(-1, E)


def rows(far, kind, gen):
    l = far.clone()
    near = torch.randn(l.shape, generator=gen)
    if kind == "odd experts near":
        l[:, 1::2] = near[:, 1::2]
    elif kind == "two groups near":
        l[:, 16:32] = near[:, 16:32]
    elif kind == "one expert near":
        l[:, 37] = near[:, 37]
    return l


def test_a_far_logit_wins_by_its_bias():
    l, bias = torch.tensor([[-90.5, 0.0]]), torch.tensor([2.0, 0.0])
    for top in (1, 2):
        w, ids = router.route(l.cuda(), top, score="sigmoid", bias=bias.cuda())
        assert ids.tolist() == [[0, 1][:top]]
    check(l, 2, score="sigmoid", bias=bias)


@pytest.mark.parametrize("kind", ["all far", "odd experts near", "two groups near", "one expert near"])
@pytest.mark.parametrize("lo, hi", [(-210, -80), (80, 210)])
@pytest.mark.parametrize("dt", TYPES)
def test_the_choice_of_far_logits(kind, lo, hi, dt):
    print("far", kind, lo, dt, flush=True)
    gen = torch.Generator().manual_seed(3)
    l = rows(sweep(lo, hi), kind, gen).to(TYPES[dt])
    small = torch.randn(E, generator=gen) * 0.05
    ahead = torch.zeros(E)
    ahead[::2] = 2.0   # of the far ones, where others are near
    masked = ahead.clone()
    masked[::4] = -math.inf
    for score in ("sigmoid", "softmax"):
        for i, bias in enumerate((small, ahead, masked, torch.zeros(E), None)):
            kw = dict(score=score, bias=bias, renormalize=i % 2 == 0, scale=2.5)
            check(l, 6, **kw)
            for best in (1, 2):
                check(l, 6, groups=8, top_groups=3, group_best=best, **kw)
