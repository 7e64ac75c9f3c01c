"""The 4-bit product with more rows than one block of rows holds (the later
blocks find the scale table in place and only wait for their own operands).
Against float64 on the CPU; tolerance as include/gemm.h gives it: half a step of
the output type, plus 2^-20 of the sum of 31 |X s|, fp16's subnormal step."""
import pytest
import torch

from dense_tiled_gemm_02_amd import w4

pytestmark = pytest.mark.gpu


def run(M, N, K, G, dtype, E=0, ids=None):
    gen = torch.Generator().manual_seed(M + N + K)
    lead = (E,) if E else ()
    x = torch.randn((M, K), generator=gen).to(dtype)
    w = torch.randint(0, 256, lead + (N, K // 2), generator=gen, dtype=torch.uint8)
    s = ((torch.rand(lead + (N, -(-K // G)), generator=gen) + 0.1) * 0.01).to(dtype)
    sc = s.double().repeat_interleave(G, -1)[..., :K]
    v = (torch.stack((w & 15, w >> 4), -1).flatten(-2).double() - 8) * sc
    xd, xc, wc, scu = x.double(), x.cuda(), w.cuda(), s.cuda()
    if E:
        ref = torch.stack([xd[m] @ v[e].t() if 0 <= e < E else torch.zeros(N).double() for m, e in enumerate(ids)])
        S = torch.stack([xd[m].abs() @ (31 * sc[e]).t() if 0 <= e < E else torch.zeros(N).double() for m, e in enumerate(ids)])
        call = lambda: w4.w4_matvec(xc, wc, scu, group=G, experts=torch.tensor(ids).cuda())
    else:
        ref, S = xd @ v.t(), xd.abs() @ (31 * sc).t()
        call = lambda: w4.w4_matvec(xc, wc, scu, group=G)
    got = call()
    acc = 2.0 ** -20 * S
    over = (got.cpu().double() - ref).abs() - (torch.finfo(dtype).eps / 2 * (ref.abs() + acc) + acc +
                                               (2.0 ** -25 if dtype == torch.float16 else 0))
    assert torch.isfinite(got).all() and over.max().item() <= 0, over.max().item()
    for _ in range(3):
        assert torch.equal(got, call())


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(33, 64, 2048), (36, 4200, 1024), (70, 100, 4096), (130, 48, 8192 + 32), (200, 17, 384)])
def test_blocks_of_rows(M, N, K, G):
    run(M, N, K, G, torch.bfloat16 if M % 2 else torch.float16)


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M,N,K,E", [(40, 96, 2048, 2), (61, 64, 1024, 3), (64, 300, 4096, 70), (90, 33, 544, 4)])
def test_blocks_of_an_experts_rows(M, N, K, E, G):
    """One expert has 17 to 20 rows (a last block of few), another more than two blocks or none."""
    ids = [0] * (17 + M % 4) + [E - 1] * (M - 17 - M % 4)
    ids[1], ids[-1] = ids[-1], -1
    run(M, N, K, G, torch.bfloat16, E, ids)


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("N,K", [(16, 128), (40, 96), (33, 1024), (600, 4096), (5000, 2080), (9000, 1152), (17000, 544)])
def test_few_rows(M, N, K, G):
    run(M, N, K, G, torch.float16 if N % 2 else torch.bfloat16)


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N,K,E", [(64, 1024, 8), (2000, 4096, 16), (700, 8192, 60), (36, 160, 64)])
def test_few_rows_of_each_expert(N, K, E, G):
    run(30, N, K, G, torch.bfloat16, E, [(7 * m * m + m) % (E + 1) for m in range(30)])


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 7, 16])
@pytest.mark.parametrize("N,K", [(4100, 32), (5000, 608), (7001, 1152), (8192, 2016)])
def test_one_workgroup_to_a_cu_and_short_k(N, K, M, G):
    run(M, N, K, G, torch.float16 if N % 2 else torch.bfloat16)
