"""The grouped product's 64-row tile whose waves share out K, against float64 on
the CPU.  Tolerance: the output's rounding, eps / 2 of the value, and 2^-20 of
the terms' magnitudes for the fp32 sum; fp16 adds half its subnormal step."""
import numpy as np
import pytest
import torch

from dense_tiled_gemm_02_amd import grouped

pytestmark = pytest.mark.gpu
FEW = dict(bm=64, bk=32)


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
    run([1, 0, 63, 64, 65, 17, 130], K, N, dtype, trans, first=5, after=20)


@pytest.mark.parametrize("trans", [False, True], ids=["kn", "nk"])
def test_more_tiles_than_workgroups(trans):
    rng = np.random.default_rng(3)
    run(rng.integers(0, 70, 120).tolist(), 72, 264, torch.bfloat16, trans)


@pytest.mark.parametrize("trans", [False, True], ids=["kn", "nk"])
def test_repeats_bit_for_bit(trans):
    lens = [2, 90, 0, 30]
    assert torch.equal(run(lens, 520, 96, torch.float16, trans), run(lens, 520, 96, torch.float16, trans))


@pytest.mark.parametrize("off", [[0, 90, 40, 120], [500, 1, 0, 0], [-7, 60, 500, 2 ** 31 - 1]], ids=str)
def test_bad_tables_stay_inside(off):
    A, B = torch.randn(120, 64).half().cuda(), torch.randn(3, 64, 64).half().cuda()
    out = torch.full((122, 64), 7.0, dtype=torch.float16, device="cuda")
    grouped.grouped_matmul(A, B, torch.tensor(off, dtype=torch.int32, device="cuda"), out=out[1:121], config=FEW)
    assert (out[0] == 7).all() and (out[121] == 7).all()


@pytest.mark.parametrize("trans", [False, True], ids=["kn", "nk"])
def test_a_prompt_over_few_experts_takes_it(trans):
    before = set(grouped._plans)
    run([30, 17, 33], 2048, 520, torch.bfloat16, trans, config=None)
    new = [grouped._plans[k] for k in grouped._plans if k not in before]
    assert new and all((p.config.bm, p.config.bk) == (64, 32) for p in new)
