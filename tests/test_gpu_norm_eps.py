"""RMS norm of bf16 rows and eps so small that the squares' mean leaves fp32's normal
range, or so large that mean + eps passes its end (GPU).

Bounds as in test_gpu_norm.py: an output's half step, and 2^-18 for fp32."""
import pytest
import torch

from dense_tiled_gemm_02_amd import norm
from test_gpu_norm import FP32, check_rows, half_step, near, rows, smallest
from test_norm import gradient

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def f32(v):
    return float(torch.tensor(v, dtype=torch.float32))


# every kind of row: of a part of a wave, a wave, several waves, read again
@pytest.mark.parametrize("K", [5, 64, 1000, 3000, 20000, 33001])
@pytest.mark.parametrize("value, eps", [(1e-22, 1e-44), (2.0 ** -75, 2.0 ** -149), (2.0 ** -64, 2.0 ** -130), (1e-30, 1e-40),
                                        (2.0 ** -60, 2.0 ** -140), (1e-19, 1e-38), (1.0, 1e-44), (2.0 ** 63, 3e38), (2.0 ** 62, 3.4e38), (1e25, 1e-44), (1e30, 1e-20)])
def test_far_eps(K, value, eps):
    print("eps", K, value, eps, flush=True)
    x = (rows(6, K, torch.float32, K).sign() * (1 + rows(6, K, torch.float32, 1).abs().clamp(max=1.0)) * value).to(BF16)
    r = (rows(6, K, torch.float32, 2) * value).to(BF16)
    x[0], r[0] = 0, 0
    x[1], r[1] = rows(1, K, BF16, 3)[0], 0   # its neighbours are not disturbed
    w = rows(1, K, torch.float32, 4)[0]
    leaves = [t.cuda().requires_grad_() for t in (x, w, r)]
    y, h = norm.rms_norm(*leaves, eps=eps)
    h64 = (x.float() + r.float()).to(BF16).double()
    assert torch.equal(h.detach().cpu().double(), h64)
    n = torch.sqrt(h64.square().mean(1, keepdim=True) + f32(eps))
    want = h64 / n * w.double()
    near(y.detach(), want, want.abs() * (half_step(BF16) + FP32) + smallest(BF16), "y")
    assert bool((y[0] == 0).all())
    q, scale, _ = norm.rms_norm_i8(leaves[0].detach(), leaves[1].detach(), leaves[2].detach(), eps=eps)
    check_rows(q, scale, want, FP32)
    # dy of the size of n: gradients that bf16 holds
    dy = (rows(6, K, torch.float32, 5) * n.clamp(1e-30, 1e18)).to(BF16)
    dh = torch.zeros(6, K, dtype=BF16)
    got = torch.autograd.grad((y, h), leaves, (dy.cuda(), dh.cuda()))
    dx, dw = gradient(dy.double(), dh.double(), h64, w.double(), f32(eps))
    u, g = (h64 / n).abs(), (dy.double() * w.double()).abs()
    size = (g + u * (g * u).mean(1, keepdim=True)) / n
    near(got[0], dx, dx.abs() * half_step(BF16) + size * FP32 + smallest(BF16), "dx")
    near(got[1], dw, (dy.double().abs() * u).sum(0) * 2.0 ** -17 + 2.0 ** -149, "dw")
