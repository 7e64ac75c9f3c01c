"""Calls that the binding remembers give what checked calls give: other data,
other addresses, other shapes, refusals, streams, devices' rules."""
import pytest
import torch

import dense_tiled_gemm_02_amd as g
from dense_tiled_gemm_02_amd import grouped, w4

pytestmark = pytest.mark.gpu


def randn(*s, dtype=torch.bfloat16):
    return torch.randn(*s, device="cuda").to(dtype)


def test_remembered_calls_see_new_data_and_addresses():
    for seed in range(3):
        torch.manual_seed(seed)
        A, B, G = randn(100, 64), randn(3, 64, 48), randn(100, 48)
        off = torch.tensor([0, 30 + seed, 60, 100], dtype=torch.int32, device="cuda")
        assert torch.equal(grouped.grouped_matmul(A, B, off),
                           grouped.grouped_matmul(A, B, off, out=torch.empty(100, 48, dtype=A.dtype, device="cuda")))
        for od in (None, torch.float32, torch.bfloat16):
            D = grouped.grouped_wgrad(A, G, off, out_dtype=od)
            assert D.dtype == (od or A.dtype)
            assert torch.equal(D, grouped.grouped_wgrad(A, G, off, out=torch.empty_like(D)))
        ids = torch.randint(-1, 5, (100,), device="cuda")
        offsets, order = grouped.group_rows(ids, 4)
        key = torch.where(ids < 0, 4, ids)
        assert torch.equal(order.long(), torch.sort(key, stable=True).indices)
        assert offsets.tolist() == [int((key < e).sum()) for e in range(5)]
        q, s, z = w4.w4_quantize(randn(2, 40, 64), 32, zeros=True)
        x, e = randn(5, 64), torch.randint(0, 2, (5,), device="cuda")
        assert torch.equal(w4.w4_matvec(x, q, s, z, 32, experts=e),
                           w4.w4_matvec(x, q, s, z, 32, experts=e, out=torch.empty(5, 40, dtype=x.dtype, device="cuda")))


def test_every_difference_that_the_checks_see_is_a_new_call():
    A, B = randn(64, 64), randn(2, 64, 64)
    off = torch.tensor([0, 20, 64], dtype=torch.int32, device="cuda")
    for _ in range(2):
        D = grouped.grouped_matmul(A, B, off)
        assert torch.equal(D, grouped.grouped_matmul(A, B.transpose(1, 2).contiguous().transpose(1, 2), off))
        for bad in (lambda: grouped.grouped_matmul(A, B, off.long()), lambda: grouped.grouped_matmul(A, B, off[:2]),
                    lambda: grouped.grouped_matmul(A, B[:, :32], off), lambda: grouped.grouped_matmul(A.cpu(), B, off),
                    lambda: grouped.grouped_matmul(A, B, off.cpu())):
            with pytest.raises(ValueError):
                bad()
        with pytest.raises(TypeError):
            grouped.grouped_matmul(A, B.half(), off)
        with pytest.raises(TypeError):
            grouped.grouped_wgrad(A, A, off, out_dtype=torch.float16)
        with pytest.raises(g.GemmError):
            grouped.group_rows(off, -1)


def test_refusals_of_a_remembered_call():
    buf = torch.zeros(2 * 64 + 8, dtype=torch.float16, device="cuda")
    w = torch.zeros(8, 32, dtype=torch.uint8, device="cuda")
    s = torch.ones(8, 1, dtype=torch.float16, device="cuda")
    good, bad = buf[:128].view(2, 64), buf[1:129].view(2, 64)
    w4.w4_matvec(good, w, s, group=64)
    for _ in range(2):
        with pytest.raises(g.GemmError):
            w4.w4_matvec(bad, w, s, group=64)
        assert (w4.w4_matvec(good, w, s, group=64) == 0).all()


def test_parameters_views_and_streams():
    A, W = randn(32, 64), torch.nn.Parameter(randn(2, 64, 64))
    off = torch.tensor([0, 16, 32], dtype=torch.int32, device="cuda")
    want = grouped.grouped_matmul(A, W.detach(), off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            got = grouped.grouped_matmul(A, W, off)
    side.synchronize()
    assert torch.equal(got, want) and not got.requires_grad
    x = A.clone().requires_grad_()
    grouped.grouped_linear(x, W, off).float().sum().backward()
    assert x.grad.shape == x.shape and W.grad.shape == W.shape


def test_more_calls_than_the_table_holds():
    A, B = randn(4200, 8), randn(1, 8, 8)
    off = torch.tensor([0, 4200], dtype=torch.int32, device="cuda")
    ones = torch.zeros(4200, dtype=torch.int32, device="cuda")
    for n in range(1, 4200):
        grouped.group_rows(ones[:n], 2)
    offsets, order = grouped.group_rows(ones, 2)
    assert offsets.tolist() == [0, 4200, 4200] and torch.equal(order, torch.arange(4200, device="cuda", dtype=torch.int32))
    assert grouped.grouped_matmul(A, B, off).shape == (4200, 8)
