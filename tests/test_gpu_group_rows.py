"""The row grouping over its launches' borders, against a stable sort."""
import pytest
import torch

from dense_tiled_gemm_02_amd import grouped

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("E", [1, 7, 64, 1023])
@pytest.mark.parametrize("R", [1023, 1025, 4096, 4097, 16384, 16385, 17408, 17409, 20479, 65537, 131072, 262144, 262145,
                               300001])
def test_sizes(R, E, dtype):
    gen = torch.Generator().manual_seed(R + E)
    ids = torch.randint(-2, E + 2, (R,), generator=gen)
    if R % 2:                                             # long runs of one id
        ids = torch.sort(ids).values
    offsets, order = grouped.group_rows(ids.to(dtype).cuda(), E)
    key = torch.where((ids >= 0) & (ids < E), ids, E)
    want = torch.sort(key, stable=True)
    assert torch.equal(order.cpu().long(), want.indices)
    assert torch.equal(offsets.cpu().long(), torch.searchsorted(want.values, torch.arange(E + 1)))


def test_ids_at_the_ends_of_their_type():
    for dtype in (torch.int32, torch.int64):
        info = torch.iinfo(dtype)
        ids = torch.tensor([info.max, 1, info.min, 0, 2, 2 ** 31 - 1, 1] * 3000, dtype=dtype)
        offsets, order = grouped.group_rows(ids.cuda(), 2)
        key = torch.where((ids >= 0) & (ids < 2), ids, 2)
        assert torch.equal(order.cpu().long(), torch.sort(key, stable=True).indices)
        assert offsets.tolist() == [0, 3000, 9000]
