"""Host side of the grouped products, the row grouping and the 4-bit product:
planning against a hand-made device, refusals of the C ABI and of the torch
binding (CPU only: no kernel is launched)."""
import ctypes

import pytest
import torch

import dense_tiled_gemm_02_amd as g
from dense_tiled_gemm_02_amd import grouped, w4
from test_abi import fake_gfx950

INVALID, UNSUPPORTED, WORKSPACE = g.GEMM_ERR_INVALID_ARG, g.GEMM_ERR_UNSUPPORTED, g.GEMM_ERR_WORKSPACE


def rows_problem(E=8, R=1000, P=512, Q=768, trans=False, **kw):
    p = g.gemm_grouped_problem()
    p.groups, p.R, p.P, p.Q = E, R, P, Q
    p.sa_r, p.sa_p = P, 1
    p.sb_g, p.sb_r, p.sb_q = P * Q, (1 if trans else Q), (P if trans else 1)
    p.sd_r = Q
    p.dtype, p.kind = g.GEMM_BF16, g.GEMM_GROUPED_ROWS
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def reduce_problem(E=8, R=1000, P=512, Q=768, **kw):
    p = rows_problem(E, R, P, Q)
    p.sb_g, p.sb_r, p.sb_q = 0, Q, 1
    p.sd_g, p.sd_r = P * Q, Q
    p.kind = g.GEMM_GROUPED_REDUCE
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def w4_problem(M=4, N=256, K=512, group=128, experts=0, **kw):
    p = g.gemm_w4_problem()
    p.M, p.N, p.K, p.group, p.experts = M, N, K, group, experts
    n = -(-K // group) if group > 0 else 0
    p.sx, p.sy, p.sw_n, p.sw_e, p.ss_n, p.ss_e, p.sz_n, p.sz_e = K, N, K // 2, N * K // 2, n, N * n, n, N * n
    p.dtype, p.id_bytes = g.GEMM_F16, 8
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def plan(p, force=None):
    return grouped.gemm_grouped_plan_create_for(p, fake_gfx950(), force)


def refused(status, call):
    with pytest.raises(g.GemmError) as e:
        call()
    assert e.value.status == status and e.value.detail


@pytest.mark.parametrize("trans", [False, True])
def test_aligned_operands_take_the_direct_tiles_and_others_the_element_wise(trans):
    assert "gemm_grouped_rows_kernel" in plan(rows_problem(trans=trans)).describe()
    assert "gemm_grouped_reduce_kernel" in plan(reduce_problem()).describe()
    for kw in (dict(P=511), dict(sa_p=2), dict(sa_r=516), dict(sa_r=504), dict(sb_g=512 * 768 + 4), dict(sa_r=0)):
        assert "any_kernel" in plan(rows_problem(trans=trans, **kw)).describe(), kw
    assert "any_kernel" in plan(rows_problem(sb_r=760)).describe()      # overlapping rows of B
    assert "any_kernel" in plan(rows_problem(Q=765)).describe()
    # B stored Q x P: only P and its strides matter, Q is free
    assert "rows_kernel" in plan(rows_problem(Q=765, trans=True)).describe()
    for kw in (dict(sb_q=0), dict(sb_r=0), dict(Q=763), dict(P=500)):
        assert "any_kernel" in plan(reduce_problem(**kw)).describe(), kw


def test_grid_covers_every_table():
    """floor(R / BM) + E + 2 rows of tiles: each of E + 2 segments has at most
    one tile that is not full."""
    for E, R in ((1, 1), (3, 1000), (64, 64), (100, 5000)):
        pl = plan(rows_problem(E=E, R=R))
        bm, bn = pl.config.bm, pl.config.bn
        assert pl.launch()[0] == (R // bm + E + 2) * -(-768 // bn)
        # the worst table: as many ragged groups as the rows allow
        ragged = min(E, R)
        most = sum(-(-n // bm) for n in [R // ragged + (i < R % ragged) for i in range(ragged)])
        assert most <= R // bm + E + 2
    pl = plan(reduce_problem(E=5))
    assert pl.launch()[0] == 5 * -(-512 // pl.config.bm) * -(-768 // pl.config.bn)


def test_forced_tiles():
    for cfg in (dict(bm=256, bn=256), dict(bm=64, bn=64), dict(bm=128, bn=128, stages=2)):
        c = plan(rows_problem(), cfg).config
        assert all(getattr(c, k) == v for k, v in cfg.items())
    assert plan(rows_problem(), dict(group_m=3, xcd_remap=2)).config.group_m == 3
    refused(UNSUPPORTED, lambda: plan(rows_problem(), dict(bm=96)))
    refused(UNSUPPORTED, lambda: plan(rows_problem(), dict(splitk=2)))
    refused(UNSUPPORTED, lambda: plan(rows_problem(), dict(kernel=3)))
    refused(INVALID, lambda: plan(rows_problem(), dict(xcd_remap=3)))


def test_grouped_problem_refusals():
    for kw in (dict(E=-1), dict(R=-1), dict(P=-1), dict(Q=-1), dict(kind=2), dict(dtype=7), dict(out=2),
               dict(accumulate=2), dict(sd_r=767), dict(sa_r=1 << 60), dict(sb_g=1 << 62)):
        refused(INVALID, lambda: plan(rows_problem(**kw)))
    for kw in (dict(dtype=g.GEMM_I8), dict(out=1), dict(accumulate=1), dict(R=1 << 31), dict(E=65536), dict(sa_r=-1),
               dict(sb_q=-8), dict(R=(1 << 31) - 1, Q=1 << 20)):
        refused(UNSUPPORTED, lambda: plan(rows_problem(**kw)))
    refused(INVALID, lambda: plan(reduce_problem(sd_g=512 * 768 - 1)))
    refused(INVALID, lambda: grouped.gemm_grouped_plan_create_for(rows_problem(), g.gemm_device_info()))
    assert g.lib().gemm_grouped_plan_create_for(None, None, None, None) == INVALID
    h = ctypes.c_void_p(1)
    assert g.lib().gemm_grouped_plan_create_for(None, None, None, ctypes.byref(h)) == INVALID and not h.value
    g.lib().gemm_grouped_plan_destroy(None)


def test_grouped_run_refusals():
    """Refused before any device call; the addresses are never read."""
    pl = plan(rows_problem(E=2, R=100))
    A, B, O, D = 1 << 20, 1 << 24, 1 << 16, 1 << 28
    run = grouped.gemm_grouped_run
    refused(INVALID, lambda: run(pl, A, B, O, None))
    refused(INVALID, lambda: run(pl, A, B, None, D))
    refused(INVALID, lambda: run(pl, None, B, O, D))
    refused(INVALID, lambda: run(pl, A, None, O, D))
    refused(INVALID, lambda: run(pl, A, B, O, A + 64))
    refused(INVALID, lambda: run(pl, A, B, O, B + 512 * 768 * 4 - 2))
    refused(INVALID, lambda: run(pl, A, B, D + 4, D))
    refused(UNSUPPORTED, lambda: run(pl, A + 1, B, O, D))
    refused(UNSUPPORTED, lambda: run(pl, A, B, O + 2, D))
    refused(UNSUPPORTED, lambda: run(plan(reduce_problem(out=1)), A, A + (1 << 26), O, D + 2))
    assert g.lib().gemm_grouped_run(None, A, B, O, D, None) == INVALID
    # nothing to write: no launch, whatever the pointers
    run(plan(rows_problem(R=0)), None, None, None, None)
    run(plan(rows_problem(Q=0, sd_r=0)), None, None, None, None)
    run(plan(reduce_problem(E=0)), None, None, None, None)


def test_group_rows_refusals():
    ws = grouped.gemm_group_rows_workspace
    assert ws(16384, 8) == 0 and ws(16385, 8) == 5 * 9 * 4
    refused(UNSUPPORTED, lambda: ws(10, 1024))
    refused(UNSUPPORTED, lambda: ws(1 << 31, 8))
    refused(INVALID, lambda: ws(-1, 8))
    run = grouped.gemm_group_rows
    I, F, O, W = 1 << 20, 1 << 24, 1 << 26, 1 << 28
    refused(INVALID, lambda: run(I, 2, 10, 4, F, O))
    refused(INVALID, lambda: run(None, 4, 10, 4, F, O))
    refused(INVALID, lambda: run(I, 4, 10, 4, None, O))
    refused(INVALID, lambda: run(I, 4, 10, 4, F, None))
    refused(UNSUPPORTED, lambda: run(I + 4, 8, 10, 4, F, O))
    refused(INVALID, lambda: run(I, 8, 10, 4, F, I + 76))
    refused(INVALID, lambda: run(I, 4, 10, 4, I + 36, O))
    refused(WORKSPACE, lambda: run(I, 4, 20000, 4, F, O))
    refused(WORKSPACE, lambda: run(I, 4, 20000, 4, F, O, W, 99))
    refused(WORKSPACE, lambda: run(I, 4, 20000, 4, F, O, W + 2, 1000))
    refused(INVALID, lambda: run(I, 4, 20000, 4, F, O, O + 8, 1000))


def test_w4_plans_and_refusals():
    make = lambda **kw: w4.gemm_w4_plan_create_for(w4_problem(**kw), fake_gfx950())
    for G in (32, 64, 128):
        assert ",%d,0,0>" % G in make(group=G).describe()
    assert "rows=32" in make(M=17).describe() and "rows=16" in make(M=17, experts=4).describe()
    for kw in (dict(M=-1), dict(N=-1), dict(experts=-1), dict(dtype=9), dict(has_zeros=2), dict(experts=2, id_bytes=2),
               dict(sy=255), dict(sw_n=1 << 60), dict(ss_n=1 << 60)):
        refused(INVALID, lambda: make(**kw))
    for kw in (dict(dtype=g.GEMM_I8), dict(group=16), dict(group=256), dict(group=0), dict(K=520), dict(sx=516),
               dict(sw_n=264), dict(experts=65536), dict(sx=-8), dict(M=1 << 31), dict(has_zeros=1, sz_n=-1)):
        refused(UNSUPPORTED, lambda: make(**kw))
    pl, px = make(has_zeros=1), make(experts=3)
    X, W, S, Z, I, Y = (1 << b for b in (20, 22, 24, 26, 27, 28))
    run = w4.gemm_w4_run
    refused(INVALID, lambda: run(pl, X, W, S, None, None, Y))
    refused(INVALID, lambda: run(pl, None, W, S, Z, None, Y))
    refused(INVALID, lambda: run(pl, X, W, S, Z, None, None))
    refused(INVALID, lambda: run(pl, X, W, S, Z, I, Y))
    refused(INVALID, lambda: run(px, X, W, S, Z, I, Y))
    refused(INVALID, lambda: run(px, X, W, S, None, None, Y))
    refused(INVALID, lambda: run(pl, X, W, S, Z, None, W + 100))
    refused(INVALID, lambda: run(pl, X, W, S, Z, None, Z + 2))
    refused(INVALID, lambda: run(px, X, W, S, None, Y + 8, Y))
    refused(UNSUPPORTED, lambda: run(pl, X + 8, W, S, Z, None, Y))
    refused(UNSUPPORTED, lambda: run(pl, X, W + 8, S, Z, None, Y))
    refused(UNSUPPORTED, lambda: run(pl, X, W, S + 1, Z, None, Y))
    refused(UNSUPPORTED, lambda: run(px, X, W, S, None, I + 4, Y))
    run(make(M=0), None, None, None, None, None, None)


def test_binding_refusals():
    z = lambda *s, dtype=torch.float16: torch.zeros(s, dtype=dtype)
    off = torch.zeros(3, dtype=torch.int32)
    gm, gw = grouped.grouped_matmul, grouped.grouped_wgrad
    for call in (lambda: gm(z(4, 8), z(2, 8, 8), off),                       # CPU tensors
                 lambda: gm(z(4, 8), z(2, 16, 8), off), lambda: gm(z(4, 8), z(8, 8), off),
                 lambda: gw(z(4, 8), z(5, 8), off), lambda: gw(z(4, 8), z(4, 8), off[:0]),
                 lambda: grouped.group_rows(torch.zeros(4, dtype=torch.int64), 2),
                 lambda: grouped.group_rows(torch.zeros(4, 2, dtype=torch.int64), 2)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gm(z(4, 8, dtype=torch.float32), z(2, 8, 8), off),
                 lambda: gm(z(4, 8), z(2, 8, 8, dtype=torch.bfloat16), off),
                 lambda: grouped.group_rows(z(4), 2)):
        with pytest.raises(TypeError):
            call()
    x, w, s = z(2, 64), z(8, 32, dtype=torch.uint8), z(8, 1)
    mv = w4.w4_matvec
    for call in (lambda: mv(x, w, s, group=64), lambda: mv(x[:, :32], w, s, group=64), lambda: mv(x, w, s, group=32),
                 lambda: mv(x, w[None], s[None], group=64), lambda: mv(x, w, s, group=0),
                 lambda: mv(x, w[None], s[None], group=64, experts=torch.zeros(3, dtype=torch.int64)),
                 lambda: mv(x.t().contiguous().t(), w, s, group=64), lambda: mv(x, w, s, group=64, out=z(2, 9)),
                 lambda: w4.w4_quantize(z(4, 40))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mv(x.float(), w, s.float(), group=64), lambda: mv(x, w.char(), s, group=64),
                 lambda: mv(x, w, s.bfloat16(), group=64), lambda: mv(x, w, s, zeros=z(8, 1), group=64),
                 lambda: mv(x, w[None], s[None], group=64, experts=z(2)), lambda: w4.w4_quantize(torch.zeros(4, 32))):
        with pytest.raises(TypeError):
            call()


def test_quantize_on_the_cpu():
    W = torch.arange(-8, 8, dtype=torch.float32).repeat(2, 4).to(torch.float16)   # 2 x 64
    q, s, z = w4.w4_quantize(W.clamp(-7, 7), group=32)
    assert z is None and (s == 1).all() and q.shape == (2, 32)
    assert q[0, 0] == 1 | 1 << 4 and q[0, 1] == 2 | 3 << 4                        # -7, -7 | -6, -5, plus 8
    q, s, z = w4.w4_quantize(W, group=64, zeros=True)
    assert (s == 1).all() and (z == 8).all() and q[0, 7] == 14 | 15 << 4
    q, s, z = w4.w4_quantize(torch.zeros(2, 32, dtype=torch.bfloat16), group=128)
    assert (q == 0x88).all() and torch.isfinite(s).all()


def test_contiguous_operands_at_any_alignment_take_chunked_loads():
    for kw in (dict(P=511), dict(sa_r=516), dict(sb_g=512 * 768 + 4), dict(sa_r=0)):
        assert "rows_odd_any_kernel" in plan(rows_problem(**kw)).describe(), kw
        assert "rows_odd_any_kernel" in plan(rows_problem(trans=True, **kw)).describe(), kw
    assert "reduce_odd_any_kernel" in plan(reduce_problem(Q=763)).describe()
    # twice-strided or shorter than a chunk: element loads
    for kw in (dict(sa_p=2), dict(P=7), dict(Q=7)):
        assert "rows_any_kernel" in plan(rows_problem(**kw)).describe(), kw
    assert "reduce_any_kernel" in plan(reduce_problem(P=7)).describe()
