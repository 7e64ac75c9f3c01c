"""Weight gradients cut into parts, and the order of the groups, against
float64 on the CPU.  Tolerance: the output's rounding, eps / 2 of the value,
and 2^-20 of the terms' magnitudes for the fp32 sums; fp16 adds half its
subnormal step."""
import numpy as np
import pytest
import torch

from dense_tiled_gemm_02_amd import grouped

pytestmark = pytest.mark.gpu


def check(got, ref, S):
    dtype, got = got.dtype, got.cpu().double()
    acc = 2.0 ** -20 * S
    bound = torch.finfo(dtype).eps / 2 * (ref.abs() + acc) + acc + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    over = (got - ref).abs() - bound
    assert torch.isfinite(got).all() and over.max().item() <= 0, over.max().item()


def inputs(R, M, N, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(R, M, generator=gen).to(dtype), torch.randn(R, N, generator=gen).to(dtype)


def reference(A, G, off):
    A, G = A.double(), G.double()
    ref = torch.stack([A[lo:max(lo, hi)].t() @ G[lo:max(lo, hi)] for lo, hi in zip(off, off[1:])])
    S = torch.stack([A[lo:max(lo, hi)].abs().t() @ G[lo:max(lo, hi)].abs() for lo, hi in zip(off, off[1:])])
    return ref, S


def is_cut(A, G, off):
    grouped.grouped_wgrad(A, G, off)
    return max(p.workspace for k, p in grouped._plans.items() if k[6] == A.shape[0] and k[7:9] == (A.shape[1], G.shape[1])) > 0


@pytest.mark.parametrize("out", [None, torch.float32])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("lens", [[12000], [0, 12000], [11999, 1], [3, 5000, 0, 6997]], ids=str)
def test_parts(lens, dtype, out):
    R, M, N = sum(lens) + 40, 72, 136     # the last rows in no group
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    A, G = inputs(R, M, N, dtype)
    a, g, o = A.cuda(), G.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda")
    ref, S = reference(A, G, off)
    first = grouped.grouped_wgrad(a, g, o, out_dtype=out)
    check(first, ref, S)
    assert torch.equal(first, grouped.grouped_wgrad(a, g, o, out_dtype=out))
    start = torch.randn(len(lens), M + 1, N + 3).to(out or dtype)
    acc = start.cuda()[:, :M, :N]
    grouped.grouped_wgrad(a, g, o, out=acc, accumulate=True)
    check(acc, ref + start[:, :M, :N].double(), S + start[:, :M, :N].double().abs())


def test_one_group_of_12000_rows_is_cut():
    A, G = inputs(12000, 264, 520, torch.bfloat16)
    assert is_cut(A.cuda(), G.cuda(), torch.tensor([0, 12000], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("off", [[0, 9000, 4000, 12000], [5000, 100, 0, 0], [-7, 6000, 50000, 2 ** 31 - 1]], ids=str)
def test_bad_tables_stay_inside(off):
    A, G = inputs(12000, 72, 136, torch.float16)
    guard = torch.full((5, 72, 136), 7.0, device="cuda")
    grouped.grouped_wgrad(A.cuda(), G.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"), out=guard[1:4])
    assert (guard[0] == 7).all() and (guard[4] == 7).all()


def test_graph_replays_with_other_tables():
    A, G = inputs(12000, 72, 136, torch.bfloat16)
    a, g = A.cuda(), G.cuda()
    off = torch.tensor([0, 4000, 12000], dtype=torch.int32, device="cuda")
    grouped.grouped_wgrad(a, g, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        D = grouped.grouped_wgrad(a, g, off)
    for table in ([0, 12000, 12000], [0, 1, 9000], [100, 8000, 11000]):
        off.copy_(torch.tensor(table, dtype=torch.int32))
        graph.replay()
        eager = grouped.grouped_wgrad(a, g, off)
        torch.cuda.synchronize()
        assert torch.equal(D, eager)
        check(D, *reference(A, G, table))


@pytest.mark.parametrize("E", [1, 7, 8, 63, 64, 65])
def test_groups_in_order_of_length(E):
    """Groups of 256 rows and more on average run longest first (up to 64)."""
    rng = np.random.default_rng(E)
    lens = rng.multinomial(300 * E, rng.dirichlet(np.full(E, 0.7)))
    lens[rng.integers(E)] += 50
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    A, G = inputs(off[-1], 128, 64, torch.bfloat16, E)
    for cfg in (dict(bm=64, bn=64), dict(bm=128, bn=128, bk=32), dict(bm=128, bn=128, bk=64)):
        D = grouped.grouped_wgrad(A.cuda(), G.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"),
                                  out_dtype=torch.float32, config=cfg)
        check(D, *reference(A, G, off))


def test_a_die_takes_its_share_of_every_group():
    """Tiles that divide by the dies (64 of them), and one column more."""
    for N in (512, 520):
        A, G = inputs(2000, 512, N, torch.float16, N)
        off = [0, 900, 900, 1500, 2000]
        D = grouped.grouped_wgrad(A.cuda(), G.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"),
                                  out_dtype=torch.float32, config=dict(bm=64, bn=64))
        check(D, *reference(A, G, off))
