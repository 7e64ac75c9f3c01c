"""The row operators and the int8 products where offsets pass 32 bits: the first,
the last and some rows between against the same rows alone, bit by bit (GPU)."""
import pytest
import torch

from dense_tiled_gemm_02_amd import i8, norm, router

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def places(R, n):
    """Runs of rows at the start, around the middle and at the end."""
    return [slice(0, n), slice(R // 2 + 1, R // 2 + 1 + n), slice(R - n, R)]


def same(a, b, what):
    assert torch.equal(a, b), what


def test_norm_and_its_gradient():
    R, K = (1 << 18) + 5, 16400   # 8.6 GB each
    x = torch.randn(1024, K, dtype=torch.bfloat16, device="cuda").repeat(R // 1024 + 1, 1)[:R]
    x[-3:] *= 3
    w = torch.randn(K, dtype=torch.bfloat16, device="cuda")
    y, h = norm.rms_norm(x, w, x)
    q, scale, h8 = norm.rms_norm_i8(x, w, x)
    v, steps = i8.i8_quantize(x)
    for at in places(R, 3):
        some = norm.rms_norm(x[at], w, x[at])
        same(y[at], some[0], "y")
        same(h[at], some[1], "h")
        for a, b in zip((q, scale, h8), norm.rms_norm_i8(x[at], w, x[at])):
            same(a[at], b, "rows of a norm")
        for a, b in zip((v, steps), i8.i8_quantize(x[at])):
            same(a[at], b, "rows")
    del y, h, q, scale, h8, v, steps
    rstd = torch.rand(R, device="cuda") + 0.5
    dx, _ = norm.rms_norm_grad(x, x, w, rstd)
    for at in places(R, 3):
        same(dx[at], norm.rms_norm_grad(x[at], x[at], w, rstd[at], need_weight=False)[0], "dx")


@pytest.mark.parametrize("K, stride", [(8192, 8192), (8190, 8195)])
def test_int8_rows(K, stride):
    M, N = (1 << 19) + 77, 96   # 4.3 GB
    X = torch.randint(-127, 128, (1000, stride), dtype=torch.int8, device="cuda").repeat(M // 1000 + 1, 1)[:M, :K]
    W = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    sx, sw = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    Y = i8.i8_matmul(X, sx, W, sw)
    for at in places(M, 40):
        same(Y[at], i8.i8_matmul(X[at], sx[at], W, sw), "rows of X")
    # the same as W, of few rows of X and of many
    for m in (3, 96):
        Y = i8.i8_matmul(W[:m], sw[:m], X, sx)
        for at in places(M, 40):
            same(Y[:, at], i8.i8_matmul(W[:m], sw[:m], X[at], sx[at]), "rows of W")


def test_int8_outputs():
    M, N, K = (1 << 18) + 9, 16500, 64   # 2^32 outputs and more
    X, W = (torch.randint(-127, 128, (n, K), dtype=torch.int8, device="cuda") for n in (M, N))
    sx, sw = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    for out in (torch.bfloat16, torch.float32):
        Y = i8.i8_matmul(X, sx, W, sw, out_dtype=out)
        for at in places(M, 40):
            same(Y[at], i8.i8_matmul(X[at], sx[at], W, sw, out_dtype=out), "outputs")
        del Y


def test_routing():
    R, E = (1 << 24) + 321, 160   # more rows than a launch takes, 2^31 logits and more
    some = torch.randn(4096, E, dtype=torch.bfloat16, device="cuda")
    logits = some.repeat(R // 4096 + 1, 1)[:R].requires_grad_()
    weights, ids = router.route(logits, 6)
    dw = torch.rand(R, 6, device="cuda")
    dl, = torch.autograd.grad(weights, logits, dw)
    for at in places(R, 50) + [slice((1 << 24) - 20, (1 << 24) + 20)]:
        part = logits.detach()[at].requires_grad_()
        w, i = router.route(part, 6)
        same(weights[at], w, "weights")
        same(ids[at], i, "ids")
        same(dl[at], torch.autograd.grad(w, part, dw[at].contiguous())[0], "gradient")
