"""Weight gradients whose groups are cut into parts: plans and refusals (CPU)."""
import ctypes

import pytest

import dense_tiled_gemm_02_amd as g
from dense_tiled_gemm_02_amd import grouped


def fake_gfx950():
    info = g.gemm_device_info()
    info.cu_count, info.xcd_count, info.lds_per_wg, info.lds_per_cu = 256, 8, 163840, 163840
    return info


def plan(E=1, R=12000, P=264, Q=520, out=1, force=None, **kw):
    p = g.gemm_grouped_problem()
    p.groups, p.R, p.P, p.Q = E, R, P, Q
    p.sa_r, p.sa_p, p.sb_r, p.sb_q, p.sd_g, p.sd_r = P, 1, Q, 1, P * Q, Q
    p.dtype, p.kind, p.out = g.GEMM_BF16, g.GEMM_GROUPED_REDUCE, out
    for k, v in kw.items():
        setattr(p, k, v)
    return grouped.gemm_grouped_plan_create_for(p, fake_gfx950(), force)


def part_rows(pl):
    return int(pl.describe().split("part_rows=")[1])


def test_few_tiles_and_many_rows_are_cut():
    pl = plan()
    q = part_rows(pl)
    assert q >= 512 and pl.workspace == (12000 // q + 1) * 264 * 520 * 4
    for whole in (plan(R=300), plan(E=64, R=16384, P=1408, Q=2048), plan(force=dict(bm=64, bn=64)), plan(Q=523, sd_r=523),
                  plan(E=0), plan(R=0)):
        assert part_rows(whole) == 0 and whole.workspace == 0
    # bounded however many groups share the rows
    for E in (1, 2, 4, 16, 64):
        assert plan(E=E, R=1 << 24, P=64, Q=64).workspace <= 256e6


def test_workspace_refusals():
    pl = plan()
    A, B, O, D, W = 1 << 30, 1 << 31, 1 << 16, 1 << 32, 1 << 33
    run = lambda ws, n: grouped.gemm_grouped_run_parts(pl, A, B, O, D, ws, n)
    need = pl.workspace
    for status, ws, n in ((4, W, need - 1), (4, W + 8, need), (1, D, need), (1, A - 64, need), (1, B + 16, need),
                          (1, O - 16, need)):
        with pytest.raises(g.GemmError) as e:
            run(ws, n)
        assert g.gemm_status_string(e.value.status) in ("GEMM_ERR_WORKSPACE", "GEMM_ERR_INVALID_ARG")
        assert (e.value.status == 1) == (status == 1)
    n = ctypes.c_size_t()
    assert g.lib().gemm_grouped_workspace(None, ctypes.byref(n)) == 1
    assert g.lib().gemm_grouped_workspace(pl.handle, None) == 1
