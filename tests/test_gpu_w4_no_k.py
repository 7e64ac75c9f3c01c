"""4-bit products over no k: zeros, whatever strides torch gives the empty
operands (a contiguous 5 x 0 tensor has rows one element apart)."""
import pytest
import torch

from dense_tiled_gemm_02_amd import w4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zp"])
@pytest.mark.parametrize("M", [1, 5, 40])
@pytest.mark.parametrize("E", [0, 3])
def test_zeros(E, M, zeros):
    N, lead = 24, ((E,) if E else ())
    x = torch.empty(M, 0, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(lead + (N, 0), dtype=torch.uint8, device="cuda")
    s = torch.empty(lead + (N, 0), dtype=torch.bfloat16, device="cuda")
    z = torch.empty(lead + (N, 0), dtype=torch.uint8, device="cuda") if zeros else None
    e = torch.arange(M, device="cuda") % 4 - 1 if E else None
    out = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):   # checked, then remembered
        assert (w4.w4_matvec(x, w, s, zeros=z, group=32, experts=e) == 0).all()
    w4.w4_matvec(x, w, s, zeros=z, group=32, experts=e, out=out[1:-1])
    assert (out[1:-1] == 0).all() and (out[0] == 7).all() and (out[-1] == 7).all()
    # a view without columns of operands that have some
    assert (w4.w4_matvec(torch.ones(M, 36, dtype=x.dtype, device="cuda")[:, 4:4], w, s, zeros=z, group=32, experts=e) == 0).all()
