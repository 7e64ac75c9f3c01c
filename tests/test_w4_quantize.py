"""w4_quantize's rounding against the groups' own ranges, from ordinary
magnitudes down to where a scale is subnormal.

The scale is stored in W's type: half a step off the range's part, 2^-11 (fp16)
or 2^-8 (bf16) of it, or half of the type's smallest step.  A value is off by half
a scale, and by up to 7 (15) of the scale's error where it would need a step
beyond the last."""
import pytest
import torch

from dense_tiled_gemm_02_amd import w4


def error_and_bound(W, group, zeros, device="cpu"):
    q, scale, zero = (t if t is None else t.cpu() for t in w4.w4_quantize(W.to(device), group=group, zeros=zeros))
    n = scale.shape[-1]
    v = torch.stack((q & 15, q >> 4), -1).flatten(-2).double().unflatten(-1, (n, group))
    z = zero.double() if zeros else torch.full(scale.shape, 8.0, dtype=torch.float64)
    w = W.double().unflatten(-1, (n, group))
    error = (w - (v - z[..., None]) * scale.double()[..., None]).abs().amax(-1)
    span = w.amax(-1).clamp(min=0) - w.amin(-1).clamp(max=0) if zeros else w.abs().amax(-1)
    steps = 15 if zeros else 7
    t = torch.finfo(W.dtype)
    off = torch.maximum(span / steps * t.eps / 2, torch.tensor(t.tiny * t.eps / 2, dtype=torch.float64))
    # the zero point is rounded as well: another half step
    return error, (1.0 if zeros else 0.5) * (span / steps + off) + steps * off


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zp"])
@pytest.mark.parametrize("dtype,least", [(torch.float16, -21), (torch.bfloat16, -130)], ids=["f16", "bf16"])
def test_small_groups(dtype, least, zeros, device):
    gen = torch.Generator().manual_seed(1)
    for power in (0, -6, -12, -13, -14, -16, least):
        W = torch.ldexp(torch.rand(6, 64, generator=gen) * 2 - 1, torch.tensor(power)).to(dtype)
        error, bound = error_and_bound(W, 32, zeros, device)
        assert (error <= bound).all(), (power, (error / bound).max().item())


def test_zeros_and_the_smallest_value():
    for dtype in (torch.float16, torch.bfloat16):
        t = torch.finfo(dtype)
        W = torch.zeros(2, 32, dtype=dtype)
        W[1, 3] = t.tiny * t.eps
        for zeros in (False, True):
            q, scale, zero = w4.w4_quantize(W, group=32, zeros=zeros)
            assert (scale > 0).all() and torch.isfinite(scale).all()
            assert (q[0] == (0x00 if zeros else 0x88)).all()
