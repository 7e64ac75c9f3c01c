"""Forward-mode derivatives: the norm and the routing have none, and say so (GPU)."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from dense_tiled_gemm_02_amd import norm, router

pytestmark = pytest.mark.gpu


def operands():
    gen = torch.Generator().manual_seed(1)
    x, r = (torch.randn(5, 64, generator=gen).bfloat16().cuda() for _ in range(2))
    return x, r, torch.randn(64, generator=gen).cuda(), torch.randn(64, generator=gen).cuda()


def calls(x, r, w, bias):
    """Each call, and the places of its operands that it is differentiable for."""
    return [(lambda x, w: norm.rms_norm(x, w), (x, w)), (lambda x, w, r: norm.rms_norm(x, w, r)[0], (x, w, r)),
            (lambda l: router.route(l, 3)[0], (x,)),
            (lambda l: router.route(l.float(), 3, score="sigmoid", bias=bias, renormalize=False)[0], (x,))]


@pytest.mark.parametrize("grad", [True, False])
def test_a_tangent_is_refused(grad):
    for fn, args in calls(*operands()):
        for remembered in (False, True):
            for leaf in (False, True):
                for i in range(len(args)):
                    given = [t.detach().clone().requires_grad_(leaf) for t in args]
                    with torch.set_grad_enabled(grad), forward_ad.dual_level():
                        given[i] = forward_ad.make_dual(given[i], torch.ones_like(given[i]))
                        with pytest.raises(RuntimeError, match="forward-mode"):
                            fn(*given)
            fn(*args)   # from here on a call that is known


def test_other_calls_inside_a_level_run():
    for fn, args in calls(*operands()):
        want = fn(*args)
        with forward_ad.dual_level():
            assert torch.equal(fn(*args), want)
            leaf = args[0].detach().clone().requires_grad_()
            got = fn(leaf, *args[1:])
            assert torch.equal(got, want) and got.requires_grad
            dual = forward_ad.make_dual(args[0], torch.ones_like(args[0]))
            assert torch.equal(fn(forward_ad.unpack_dual(dual).primal, *args[1:]), want)


def test_a_bias_moves_the_choice_alone():
    x, _, _, bias = operands()
    want = router.route(x, 3, score="sigmoid", bias=bias)
    with forward_ad.dual_level():
        got = router.route(x, 3, score="sigmoid", bias=forward_ad.make_dual(bias, torch.ones_like(bias)))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert forward_ad.unpack_dual(got[0]).tangent is None


def test_a_tangent_of_an_outputs_gradient_is_refused():
    for fn, args in calls(*operands()):
        leaves = [t.detach().clone().requires_grad_() for t in args]
        out = fn(*leaves)
        want = torch.autograd.grad(out, leaves, torch.ones_like(out), retain_graph=True)
        with forward_ad.dual_level():
            dual = forward_ad.make_dual(torch.ones_like(out), torch.ones_like(out))
            with pytest.raises(RuntimeError, match="forward-mode"):
                torch.autograd.grad(out, leaves, dual, retain_graph=True)
            for a, b in zip(torch.autograd.grad(out, leaves, torch.ones_like(out)), want):
                assert torch.equal(a, b)
