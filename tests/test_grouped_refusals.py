"""Arguments that the torch calls refuse by name (CPU)."""
import pytest
import torch

from dense_tiled_gemm_02_amd import grouped, w4


def z(*s, dtype=torch.float16):
    return torch.zeros(s, dtype=dtype)


def test_an_offset_table_without_a_dimension():
    with pytest.raises(ValueError):
        grouped.grouped_wgrad(z(4, 8), z(4, 8), torch.tensor(3, dtype=torch.int32))


@pytest.mark.parametrize("group", [0, -32])
def test_no_group_to_quantize_by(group):
    with pytest.raises(ValueError):
        w4.w4_quantize(z(4, 64), group=group)


def test_nothing_to_quantize():
    with pytest.raises(ValueError):
        w4.w4_quantize(z(64)[0], group=32)
    q, scale, zero = w4.w4_quantize(z(4, 0), group=32)
    assert q.shape == (4, 0) and scale.shape == (4, 0) and zero is None
