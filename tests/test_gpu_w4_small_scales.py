"""4-bit products whose scales are subnormal.  X holds small integers, so a sum is
an integer of few bits times a power of two: the products have to be exact."""
import pytest
import torch

from dense_tiled_gemm_02_amd import w4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 7, 20])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype,power", [(torch.float16, -20), (torch.float16, -24), (torch.bfloat16, -130),
                                         (torch.bfloat16, -133)], ids=str)
def test_exact(dtype, power, group, M):
    gen = torch.Generator().manual_seed(M)
    N, K = 40, 160
    x = torch.zeros(M, K)
    x[:, torch.randperm(K, generator=gen)[:16]] = torch.randint(-2, 3, (M, 16), generator=gen).float()   # sums to 256 at most
    w = torch.randint(0, 256, (N, K // 2), generator=gen, dtype=torch.uint8)
    scale = torch.full((N, -(-K // group)), 2.0 ** power, dtype=torch.float64).to(dtype)
    assert (scale.double() == 2.0 ** power).all()
    v = torch.stack((w & 15, w >> 4), -1).flatten(-2).double() - 8
    want = x.double() @ v.t() * 2.0 ** power
    got = w4.w4_matvec(x.to(dtype).cuda(), w.cuda(), scale.cuda(), group=group)
    assert torch.equal(got.cpu().double(), want)
