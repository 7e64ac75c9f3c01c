"""int8 products with scales: what they refuse, and which kernel a problem takes (CPU)."""
import pytest
import torch

import dense_tiled_gemm_02_amd as g
from dense_tiled_gemm_02_amd import i8
from test_abi import fake_gfx950

A = 1 << 30
INVALID, UNSUPPORTED = g.GEMM_ERR_INVALID_ARG, g.GEMM_ERR_UNSUPPORTED


def problem(M=128, N=256, K=512, **kw):
    p = g.gemm_i8_problem()
    p.M, p.N, p.K, p.sx, p.sw, p.sy = M, N, K, K, K, N
    p.out, p.has_bias = g.GEMM_BF16, 1
    for name, v in kw.items():
        setattr(p, name, v)
    return p


def plan(**kw):
    return i8.gemm_i8_plan_create_for(problem(**kw), fake_gfx950())


def refused(status, fn):
    with pytest.raises(g.GemmError) as e:
        fn()
    assert e.value.status == status, e.value


@pytest.mark.parametrize("status, change", [
    (INVALID, dict(M=-1)), (INVALID, dict(N=-1)), (INVALID, dict(K=-1)), (INVALID, dict(out=g.GEMM_I8)),
    (INVALID, dict(out=9)), (INVALID, dict(has_bias=2)), (INVALID, dict(sy=255)), (INVALID, dict(sx=1 << 60)),
    (UNSUPPORTED, dict(K=1 << 17)), (UNSUPPORTED, dict(M=(1 << 27) + 1)), (UNSUPPORTED, dict(N=(1 << 27) + 1)),
    (UNSUPPORTED, dict(M=1 << 20, N=1 << 16)), (UNSUPPORTED, dict(sx=-1)), (UNSUPPORTED, dict(sw=-16)),
    (UNSUPPORTED, dict(sy=-1)),
])
def test_refused_problems(status, change):
    refused(status, lambda: plan(**change))


@pytest.mark.parametrize("status, change", [
    (INVALID, dict(X=None)), (INVALID, dict(x_scale=None)), (INVALID, dict(W=None)), (INVALID, dict(w_scale=None)),
    (INVALID, dict(bias=None)), (INVALID, dict(Y=None)), (UNSUPPORTED, dict(Y=6 * A + 1)), (UNSUPPORTED, dict(x_scale=2 * A + 2)),
    (UNSUPPORTED, dict(w_scale=4 * A + 1)), (UNSUPPORTED, dict(bias=5 * A + 1)), (INVALID, dict(Y=A)), (INVALID, dict(Y=3 * A + 8)),
    (INVALID, dict(Y=2 * A)), (INVALID, dict(Y=4 * A)), (INVALID, dict(Y=5 * A)),
])
def test_refused_addresses(status, change):
    p = plan()
    args = dict(X=A, x_scale=2 * A, W=3 * A, w_scale=4 * A, bias=5 * A, Y=6 * A)
    args.update(change)
    refused(status, lambda: i8.gemm_i8_run(p, *args.values()))


def test_more_refusals():
    refused(INVALID, lambda: i8.gemm_i8_run(plan(has_bias=0), A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A))
    refused(INVALID, lambda: i8.gemm_i8_plan_create_for(problem(), g.gemm_device_info()))
    assert g.lib().gemm_i8_run(None, A, A, A, A, A, A, None) == INVALID
    assert g.lib().gemm_i8_plan_create_for(None, None, None) == INVALID
    i8.gemm_i8_run(plan(M=0), None, None, None, None, None, None)
    i8.gemm_i8_run(plan(N=0), None, None, None, None, None, None)


def test_sizes_at_the_limits_plan():
    for kw in (dict(K=(1 << 17) - 1), dict(K=(1 << 17) - 16), dict(M=1 << 27, N=256), dict(N=1 << 27, M=256, sy=1 << 27), dict(K=0)):
        assert plan(**kw).describe()


@pytest.mark.parametrize("kernel, change", [
    ("gemm_i8s_kernel<256,256,64,", dict(M=4096, N=4096, K=4096)),
    ("gemm_i8s_mixed_kernel<", dict(M=4096, N=14336, K=4096)), ("gemm_i8s_kernel<64,64,64,", dict(M=256, N=4096, K=4096)),
    ("gemm_i8s_kernel<128,128,64,", dict(M=2048, N=2048, K=2048)), ("gemm_i8s_kernel<256,128,64,", dict(M=512, N=14336, K=4096)),
    ("i8_few_kernel<1,1,", dict(M=1, N=4096, K=4096)), ("i8_few_kernel<1,1,", dict(M=64, N=1024, K=1024)),
    ("i8_few_kernel<1,2,", dict(M=16, N=8192, K=8192)), ("i8_few_kernel<1,4,", dict(M=1, N=28672, K=4096)),
    ("i8_few_kernel<2,2,", dict(M=32, N=8192, K=8192)), ("i8_few_kernel<2,4,", dict(M=32, N=28672, K=4096)),
    ("i8_few_kernel<4,2,", dict(M=64, N=8192, K=8192)), ("i8_few_kernel<4,2,", dict(M=128, N=4096, K=4096)),
    ("i8_any_kernel", dict(K=500)), ("i8_any_kernel", dict(sx=520)), ("i8_any_kernel", dict(sw=513)), ("i8_any_kernel", dict(K=0)),
    ("i8_any_kernel", dict(M=1, N=64, K=17)),
    # rows so far apart that 32-bit offsets of a tile would not reach them
    ("i8_any_kernel", dict(M=4096, N=4096, K=4096, sx=1 << 27)),
])
def test_which_kernel(kernel, change):
    kw = dict(change)
    if "M" in kw and "K" in kw:
        kw.setdefault("sy", kw["N"])
        kw.setdefault("sx", kw["K"])
        kw.setdefault("sw", kw["K"])
    assert kernel in plan(**kw).describe(), plan(**kw).describe()


def test_torch_calls_refuse_by_name():
    x, w = torch.zeros(3, 32, dtype=torch.int8), torch.zeros(5, 32, dtype=torch.int8)
    sx, sw = torch.ones(3), torch.ones(5)
    good = dict(X=x, x_scale=sx, W=w, w_scale=sw)
    for error, change in [(TypeError, dict(X=x.short())), (TypeError, dict(W=w.to(torch.uint8))), (TypeError, dict(out_dtype=torch.int32)),
                          (ValueError, dict(X=x[0])), (ValueError, dict(X=x[:, :31])), (ValueError, dict(W=w.t())),
                          (ValueError, dict(X=torch.zeros(32, 3, dtype=torch.int8).t())), (TypeError, dict(x_scale=sx.half())),
                          (ValueError, dict(x_scale=sx[:2])), (ValueError, dict(w_scale=torch.ones(1).expand(5))),
                          (TypeError, dict(w_scale=sw.double())), (TypeError, dict(bias=torch.zeros(5))),
                          (ValueError, dict(bias=torch.zeros(4, dtype=torch.bfloat16))),
                          (ValueError, dict(out=torch.zeros(3, 4))), (ValueError, dict(out=torch.zeros(5, 3).t())),
                          (TypeError, dict(out=torch.zeros(3, 5, dtype=torch.int32))), (ValueError, {})]:
        with pytest.raises(error):
            i8.i8_matmul(**{**good, **change})


def test_strides_past_any_memory_take_no_offsets_of_32_bits():
    for M, N, K in ((2, 2, 4096), (300, 2, 4096)):
        for change in (dict(sx=1 << 59), dict(sw=1 << 59), dict(sx=1 << 56), dict(sw=1 << 56)):
            if M > 16 and "sx" in change:
                continue   # reaches past 2^60
            assert "i8_any_kernel" in plan(M=M, N=N, K=K, **{"sx": K, "sw": K, "sy": N, **change}).describe()
