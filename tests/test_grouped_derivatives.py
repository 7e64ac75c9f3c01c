"""First and second derivatives of grouped_linear against differences, in
float64 on the CPU: plain products without a graph, as the kernels' results
are, stand in for the two operators that it is made of."""
import pytest
import torch

from dense_tiled_gemm_02_amd import grouped


def segments(offsets):
    o = offsets.tolist()
    return list(zip(o, o[1:]))


@torch.no_grad()
def matmul(A, B, offsets):
    D = A.new_zeros(A.shape[0], B.shape[2])
    for g, (lo, hi) in enumerate(segments(offsets)):
        D[lo:hi] = A[lo:hi] @ B[g]
    return D


@torch.no_grad()
def wgrad(A, G, offsets):
    return torch.stack([A[lo:hi].t() @ G[lo:hi] for lo, hi in segments(offsets)])


@pytest.fixture
def layer(monkeypatch):
    monkeypatch.setattr(grouped, "grouped_matmul", matmul)
    monkeypatch.setattr(grouped, "grouped_wgrad", wgrad)
    torch.manual_seed(0)
    offsets = torch.tensor([1, 4, 4, 8], dtype=torch.int32)   # an empty group, rows of no group at both ends
    x = torch.randn(9, 3, dtype=torch.float64, requires_grad=True)
    w = torch.randn(3, 3, 2, dtype=torch.float64, requires_grad=True)
    return x, w, offsets


@pytest.mark.parametrize("trans", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("which", ["x", "w", "both"])
def test_against_differences(layer, which, trans):
    x, w, offsets = layer
    if which != "both":
        (w if which == "x" else x).requires_grad_(False)
    fn = lambda x, w: grouped.grouped_linear(x, (w.transpose(1, 2).contiguous().transpose(1, 2) if trans else w), offsets)
    assert torch.autograd.gradcheck(fn, (x, w))
    if which == "both":   # a product of x and w: twice by x or by w alone is zero
        assert torch.autograd.gradgradcheck(fn, (x, w))


def test_penalty_on_the_input_gradient(layer):
    """The use in which constant first gradients went unnoticed: another term of
    the loss keeps it differentiable."""
    x, w, offsets = layer

    def loss(linear):
        y = linear(x, w)
        dx, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
        return torch.autograd.grad(y.square().sum() + dx.square().sum(), (x, w))

    plain = lambda x, w: torch.cat([x[:1] @ (0 * w[0])] + [x[lo:hi] @ w[g] for g, (lo, hi) in enumerate(segments(offsets))]
                                   + [x[8:] @ (0 * w[0])])
    for got, want in zip(loss(lambda x, w: grouped.grouped_linear(x, w, offsets)), loss(plain)):
        # sums of about 10 terms in float64
        assert torch.allclose(got, want, rtol=1e-12, atol=1e-12)


def test_third_derivative(layer):
    x, w, offsets = layer
    w.requires_grad_(False)

    def slope(x):
        y = grouped.grouped_linear(x, w, offsets)
        return torch.autograd.grad((y ** 3).sum(), x, create_graph=True)[0]
    assert torch.autograd.gradgradcheck(slope, (x,))
