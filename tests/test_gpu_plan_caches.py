"""The torch calls keep a bounded number of plans: a plan per row count would
otherwise pile up where row counts vary.  Calls give the same results after
their plans are dropped, by the plan caches and by the binding."""
import gc
import weakref

import pytest
import torch

import dense_tiled_gemm_02_amd as g
import dense_tiled_gemm_02_amd.mx as mx
from dense_tiled_gemm_02_amd import grouped, w4

pytestmark = pytest.mark.gpu
MOST = 4096
COUNTS = range(1, MOST + 60)


@pytest.fixture(autouse=True)
def fresh(monkeypatch):
    for m in (grouped, w4, mx):
        monkeypatch.setattr(m, "_plans", {})


def small(*s):
    return torch.randint(-1, 2, s, device="cuda").half()


@pytest.mark.parametrize("plain", [True, False], ids=["remembered", "checked"])
def test_grouped_products(plain):
    A, B, off = small(COUNTS[-1], 8), small(2, 8, 8), torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
    out = torch.empty(COUNTS[-1], 8, dtype=A.dtype, device="cuda")
    run = lambda n: grouped.grouped_matmul(A[:n], B, off, out=None if plain else out[:n])
    first = run(7).clone()
    plan = weakref.ref(next(iter(grouped._plans.values())))
    for n in COUNTS:
        run(n)
    assert 0 < len(grouped._plans) <= MOST
    assert torch.equal(run(7), first) and torch.equal(first[0], (A[0].float() @ B[0].float()).half())
    g.binding().forget()
    gc.collect()
    assert plan() is None


@pytest.mark.parametrize("plain", [True, False], ids=["remembered", "checked"])
def test_4_bit_products(plain):
    x, (q, s, _) = small(COUNTS[-1], 32), w4.w4_quantize(small(8, 32), 32)
    out = torch.empty(COUNTS[-1], 8, dtype=x.dtype, device="cuda")
    run = lambda n: w4.w4_matvec(x[:n], q, s, group=32, out=None if plain else out[:n])
    first = run(7).clone()
    plan = weakref.ref(next(iter(w4._plans.values())))
    for n in COUNTS:
        run(n)
    assert 0 < len(w4._plans) <= MOST
    assert torch.equal(run(7), first)
    g.binding().forget()
    gc.collect()
    assert plan() is None


def test_block_scaled_products():
    A = torch.full((COUNTS[-1], 32), 0x38, dtype=torch.uint8, device="cuda")   # E4M3 1.0
    S = torch.full((COUNTS[-1], 4), 127, dtype=torch.uint8, device="cuda")     # E8M0 1.0, rows of 4 bytes
    run = lambda n: mx.mx_matmul(A[:n], S[:n], A[:8], S[:8], 32, "e4m3")
    run(7)
    plan = weakref.ref(next(iter(mx._plans.values())))
    for n in COUNTS:
        run(n)
    assert 0 < len(mx._plans) <= MOST
    assert (run(7) == 32).all()
    gc.collect()
    assert plan() is None
