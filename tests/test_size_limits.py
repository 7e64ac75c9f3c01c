"""Sizes next to 2^31 (CPU).  Kernels round the contraction up to whole steps in 32
bits, where a sum past 2^31 wraps: no steps are taken and the output is zero; the
4-bit kernel counts its rows up in the same way, without end.  No planner takes
such sizes."""
import pytest

import dense_tiled_gemm_02_amd as g
from dense_tiled_gemm_02_amd import grouped, w4
from test_abi import fake_gfx950
from test_grouped import reduce_problem, refused, rows_problem, w4_problem

MOST = (1 << 31) - 4096


def dense(M, N, K, dtype):
    return g.gemm_plan_create_for(g.problem(M, N, K, dtype), fake_gfx950())


def small_w4(**kw):
    size = dict(M=1, N=1, K=32, sx=0, sy=1, sw_n=0)
    size.update(kw)
    return w4.gemm_w4_plan_create_for(w4_problem(**size), fake_gfx950())


def grouped_rows(**kw):
    size = dict(E=1, R=1, P=1, Q=1, sa_r=1, sb_r=1, sd_r=1)
    size.update(kw)
    if "Q" in kw:
        size.update(sb_r=kw["Q"], sd_r=kw["Q"])
    if "P" in kw:
        size.update(sa_r=kw["P"])
    return grouped.gemm_grouped_plan_create_for(rows_problem(**size), fake_gfx950())


def grouped_reduce(**kw):
    size = dict(E=1, R=1, P=1, Q=1)
    size.update(kw)
    return grouped.gemm_grouped_plan_create_for(reduce_problem(**size), fake_gfx950())


CASES = ([("dense K %d" % t, (lambda n, t=t: dense(1, 1, n, t))) for t in (g.GEMM_F16, g.GEMM_BF16)]
         + [("w4 " + d, (lambda n, d=d: small_w4(**{d: n}))) for d in "MNK"]
         + [("rows " + d, (lambda n, d=d: grouped_rows(**{d: n}))) for d in "RPQ"]
         + [("reduce " + d, (lambda n, d=d: grouped_reduce(**{d: n}))) for d in "RPQ"])


@pytest.mark.parametrize("make", [c[1] for c in CASES], ids=[c[0] for c in CASES])
def test_sizes_next_to_2_31(make):
    make(MOST)
    for n in (MOST + 32, (1 << 31) - 32):
        refused(g.GEMM_ERR_UNSUPPORTED, lambda: make(n))
