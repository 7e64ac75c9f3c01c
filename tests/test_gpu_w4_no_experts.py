"""4-bit products through experts of which there are none: zeros, in the order
of the stream that they are asked for on."""
import pytest
import torch

from dense_tiled_gemm_02_amd import w4

pytestmark = pytest.mark.gpu


def operands(M=5, N=24, K=64):
    x = torch.randn(M, K, device="cuda").half()
    w = torch.zeros(0, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(0, N, K // 32, dtype=torch.float16, device="cuda")
    return x, w, s, torch.zeros(M, dtype=torch.int64, device="cuda")


def test_zeros():
    x, w, s, e = operands()
    y = w4.w4_matvec(x, w, s, group=32, experts=e)
    assert y.shape == (5, 24) and y.dtype == x.dtype and (y == 0).all()


@pytest.mark.parametrize("as_handle", [False, True], ids=["stream", "handle"])
def test_on_the_given_stream(as_handle):
    x, w, s, e = operands()
    a = torch.randn(4096, 4096, device="cuda").bfloat16()
    out = torch.empty(5, 24, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):   # milliseconds of work, and then the values that the zeros have to replace
        for _ in range(20):
            a @ a
        out.fill_(7.0)
    y = w4.w4_matvec(x, w, s, group=32, experts=e, out=out, stream=side.cuda_stream if as_handle else side)
    assert y is out
    side.synchronize()
    assert (out == 0).all()
