"""The grouped product's tile for few rows per group against float64 on the CPU.
Tolerance: the output's rounding, eps / 2 of the value, and 2^-20 of the terms'
magnitudes for the fp32 sum; fp16 adds half its subnormal step."""
import numpy as np
import pytest
import torch

from dense_tiled_gemm_02_amd import grouped

pytestmark = pytest.mark.gpu
FEW = dict(bm=16)


def check(got, ref, S):
    dtype, got = got.dtype, got.cpu().double()
    acc = 2.0 ** -20 * S
    bound = torch.finfo(dtype).eps / 2 * (ref.abs() + acc) + acc + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    over = (got - ref).abs() - bound
    assert torch.isfinite(got).all() and over.max().item() <= 0, over.max().item()


def framed(rows, cols, stride, dtype, seed):
    """rows x cols inside NaN, and the clean values."""
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)).to(dtype)
    buf = torch.full((rows + 2, stride), float("nan"), dtype=dtype)
    buf[1:rows + 1, :cols] = x
    return x, buf.cuda()[1:rows + 1, :cols]


def run(lens, K, N, dtype, trans, config=FEW, first=0, after=0):
    off = np.concatenate([[first], first + np.cumsum(lens)]).tolist()
    R, E = off[-1] + after, len(lens)
    A, a = framed(R, K, K + 8, dtype, 1)
    rows, cols = (N, K) if trans else (K, N)
    B, b = framed(E * rows, cols, cols + 16, dtype, 2)
    B, b = B.unflatten(0, (E, rows)), b.unflatten(0, (E, rows))
    if trans:
        B, b = B.transpose(1, 2), b.transpose(1, 2)
    out = torch.full((R + 2, N + 4), 7.0, dtype=dtype, device="cuda")
    D = grouped.grouped_matmul(a, b, torch.tensor(off, dtype=torch.int32, device="cuda"), out=out[1:R + 1, 2:N + 2],
                               config=config)
    ref = torch.zeros(R, N, dtype=torch.float64)
    S = torch.zeros_like(ref)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        ref[lo:hi] = A[lo:hi].double() @ B[e].double()
        S[lo:hi] = A[lo:hi].double().abs() @ B[e].double().abs()
    check(D, ref, S)
    frame = out.clone()
    frame[1:R + 1, 2:N + 2] = 7.0
    assert (frame == 7.0).all()
    return D.clone()


@pytest.mark.parametrize("trans", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("K,N", [(8, 8), (32, 64), (40, 72), (248, 32), (264, 136), (1000, 40), (2056, 200)])
def test_shapes(K, N, dtype, trans):
    run([1, 0, 3, 16, 17, 2, 40], K, N, dtype, trans, first=5, after=20)


@pytest.mark.parametrize("trans", [False, True], ids=["kn", "nk"])
def test_more_tiles_than_workgroups(trans):
    rng = np.random.default_rng(3)
    run(rng.integers(0, 5, 200).tolist(), 72, 264, torch.bfloat16, trans)


@pytest.mark.parametrize("trans", [False, True], ids=["kn", "nk"])
def test_repeats_bit_for_bit_and_k_of_zero(trans):
    lens = [2, 9, 0, 30]
    assert torch.equal(run(lens, 520, 96, torch.float16, trans), run(lens, 520, 96, torch.float16, trans))
    off = torch.tensor([0, 3, 7], dtype=torch.int32, device="cuda")
    A = torch.empty(7, 0, dtype=torch.float16, device="cuda")
    B = torch.empty(2, 0, 64, dtype=torch.float16, device="cuda")
    assert (grouped.grouped_matmul(A, B, off) == 0).all()


@pytest.mark.parametrize("off", [[0, 9, 4, 12], [50, 1, 0, 0], [-7, 6, 500, 2 ** 31 - 1]], ids=str)
def test_bad_tables_stay_inside(off):
    A, B = torch.randn(12, 64).half().cuda(), torch.randn(3, 64, 64).half().cuda()
    out = torch.full((14, 64), 7.0, dtype=torch.float16, device="cuda")
    grouped.grouped_matmul(A, B, torch.tensor(off, dtype=torch.int32, device="cuda"), out=out[1:13], config=FEW)
    assert (out[0] == 7).all() and (out[13] == 7).all()


def test_decode_batches_take_it():
    A, B = torch.randn(16, 1024).half().cuda(), torch.randn(8, 512, 1024).half().cuda().transpose(1, 2)
    off = torch.arange(0, 17, 2, dtype=torch.int32, device="cuda")
    before = set(grouped._plans)
    grouped.grouped_matmul(A, B, off)
    new = [grouped._plans[k] for k in grouped._plans if k not in before]
    assert all(p.config.bm == 16 for p in new)
