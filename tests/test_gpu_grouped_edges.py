"""Calls that have to reach the kernel they are meant for: the plan of the call
itself is looked at.  Two-size launches over ragged columns and rows, whose last
round cuts tiles that hang over both edges, against the launch of one size (bit
for bit) and against float64 (test_gpu_grouped_mixed.check)."""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_02_amd as g
from dense_tiled_gemm_02_amd import grouped
from test_gpu_grouped_mixed import check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def fresh(monkeypatch):
    monkeypatch.setattr(grouped, "_plans", {})
    g.binding().forget()


def only_plan():
    plan, = grouped._plans.values()
    return plan


def cut_tiles(lens, N, first, after, cus):
    """Whole tiles that the last round cuts in four (the rule of the kernel)."""
    rows = [first] + list(lens) + [after]
    wholes = sum((r + 127) // 256 for r in rows) * -(-N // 256)
    smalls = sum(1 <= r % 256 <= 128 for r in rows) * -(-N // 128)
    cut = wholes % cus
    return cut if 4 * cut + smalls <= cus else 0


@pytest.mark.parametrize("trans", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("lens,N", [([4100], 4104), ([8200], 2200), ([7000, 3], 2312), ([3000, 3000, 3000, 200], 1928),
                                    ([2049, 2200, 2300], 2312), ([2500, 2500], 3336)], ids=str)
def test_ragged_edges_of_the_two_size_launch(lens, N, trans):
    first, after, K = 3, 150, 1000
    dtype = torch.float16 if trans else torch.bfloat16
    assert cut_tiles(lens, N, first, after, g.gemm_device_query().cu_count) > 0
    off = np.concatenate([[first], first + np.cumsum(lens)]).tolist()
    R = off[-1] + after
    A = torch.randn(R, K, device="cuda").to(dtype)
    shape = (len(lens), N, K) if trans else (len(lens), K, N)
    B = torch.randn(shape, device="cuda").to(dtype)
    B = B.transpose(1, 2) if trans else B
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    # an output that no tile writes stays NaN, and the frame has to
    frame = torch.full((R + 2, N), float("nan"), dtype=dtype, device="cuda")
    grouped.grouped_matmul(A, B, o, out=frame[1:-1])
    assert "rows_mixed_kernel" in only_plan().describe()
    assert torch.isnan(frame[0]).all() and torch.isnan(frame[-1]).all()
    assert torch.equal(frame[1:-1], grouped.grouped_matmul(A, B, o, config=dict(bm=256, bn=256)))
    check(lens, K, N, dtype, trans, first=first, after=after)


def test_a_large_product_takes_two_sizes():
    A, B = torch.randn(4000, 1024, device="cuda").half(), torch.randn(3, 1024, 2048, device="cuda").half()
    grouped.grouped_matmul(A, B, torch.tensor([0, 1000, 2000, 4000], dtype=torch.int32, device="cuda"))
    assert "rows_mixed_kernel" in only_plan().describe()


def test_a_decode_batch_takes_16_row_tiles():
    A, B = torch.randn(16, 1024).half().cuda(), torch.randn(8, 512, 1024).half().cuda().transpose(1, 2)
    grouped.grouped_matmul(A, B, torch.arange(0, 17, 2, dtype=torch.int32, device="cuda"))
    assert only_plan().config.bm == 16 and "rows_few_kernel" in only_plan().describe()
