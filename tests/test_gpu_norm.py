"""RMS norm, its gradients and rows in 8 bits against 64 bits (GPU).

Tolerances.  u is half a step of the output's type relative to the value, the
one rounding of an output.  In fp32 (steps of 2^-24): a sum of K squares goes
through at most 50 additions in a row for the sizes here (up to 5 chunks of 8 a
thread, then 10 across threads), its square root halves that, and a division and two products follow:
64 x 2^-24 = 2^-18 covers all of them."""
import pytest
import torch

from dense_tiled_gemm_02_amd import i8, norm
from test_norm import gradient

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
FP32 = 2.0 ** -18
# every number of threads and chunks to a row, one value more and less, and rows read again
WIDTHS = [1, 2, 7, 8, 9, 15, 127, 128, 129, 500, 512, 513, 1000, 1024, 1025, 2048, 2049, 4095, 4096, 4097, 8192, 8200, 16384,
          16385, 20001, 32768, 33001]
EPS = 1e-5


def half_step(t):
    return torch.finfo(t).eps / 2


def smallest(t):
    return torch.finfo(t).tiny * torch.finfo(t).eps


def rows(R, K, dt, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(R, K, generator=gen) * scale).to(dt)


def near(got, ref, bound, what=""):
    got, ref = got.double().cpu(), ref.double()
    off = (got - ref).abs()
    assert bool((off <= bound).all()), "%s off by %.3g where %.3g is allowed" % (
        what, off[off > bound].max(), bound[off > bound].min() if torch.is_tensor(bound) else bound)


def check_y(y, h, w):
    """y of the stream h (CPU tensors of the call)."""
    h64 = h.double()
    ref = h64 * w.double() / torch.sqrt(h64.square().mean(1, keepdim=True) + EPS)
    near(y, ref, ref.abs() * (half_step(y.dtype) + FP32) + smallest(y.dtype), "y")


def check_rows(q, scale, v, fp32):
    """q and scale of the rows v in 64 bits, which the kernel had to within fp32 x |v|."""
    q, scale = q.cpu(), scale.cpu()
    most = v.abs().amax(1)
    near(scale, most / 127, most / 127 * (fp32 + 2.0 ** -23) + 2.0 ** -149, "scale")
    assert int(q.abs().max()) <= 127
    s = scale.double()[:, None]
    # half a step, the values' own error, and the quotient's rounding of up to 127 x 2^-24 steps
    near(q.double() * s, v, s * (0.5 + 127 * 2.0 ** -24) + v.abs() * fp32 + 1e-300, "values")


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("dt", TYPES)
def test_norm(K, dt):
    print("norm", K, dt, flush=True)
    R = 37 if K <= 1024 else 3
    for residual, wide in ((False, False), (True, True), (True, False)):
        x, r = rows(R, K, TYPES[dt], K), rows(R, K, TYPES[dt], K + 1, 3.0)
        w = rows(1, K, torch.float32 if wide else TYPES[dt], 5)[0]
        if residual:
            y, h = norm.rms_norm(x.cuda(), w.cuda(), r.cuda(), eps=EPS)
            want = (x.float() + r.float()).to(x.dtype)
            assert torch.equal(h.cpu(), want)
        else:
            y, want = norm.rms_norm(x.cuda(), w.cuda(), eps=EPS), x
        assert y.dtype == x.dtype and y.shape == x.shape
        check_y(y, want, w)


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("dt", TYPES)
def test_norm_i8(K, dt):
    print("norm_i8", K, dt, flush=True)
    R = 37 if K <= 1024 else 3
    x, r, w = rows(R, K, TYPES[dt], K), rows(R, K, TYPES[dt], K + 1), rows(1, K, torch.float32, 6)[0]
    q, scale, h = norm.rms_norm_i8(x.cuda(), w.cuda(), r.cuda(), eps=EPS)
    h = h.cpu()
    assert torch.equal(h, (x.float() + r.float()).to(x.dtype))
    h64 = h.double()
    check_rows(q, scale, h64 * w.double() / torch.sqrt(h64.square().mean(1, keepdim=True) + EPS), FP32)
    assert len(norm.rms_norm_i8(x.cuda(), w.cuda(), eps=EPS)) == 2


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("dt", TYPES)
def test_quantize(K, dt):
    """Exactly the steps of the stored scale: the same fp32 operations on the CPU."""
    print("quantize", K, dt, flush=True)
    x = rows(37 if K <= 1024 else 3, K, TYPES[dt], K)
    x[0] *= 2.0 ** -14
    q, scale = i8.i8_quantize(x.cuda())
    s = x.float().abs().amax(1) / 127
    assert torch.equal(scale.cpu(), s)
    want = torch.where(s[:, None] > 0, x.float() / s[:, None], torch.zeros(1)).round().clamp(-127, 127)
    assert torch.equal(q.cpu().float(), want)
    check_rows(q, scale, x.double(), 0.0)


@pytest.mark.parametrize("K", [1, 7, 128, 200, 1000, 1024, 2048, 3001, 4096, 8192, 9000, 16384, 20001])
@pytest.mark.parametrize("dt", TYPES)
def test_gradients(K, dt):
    print("gradients", K, dt, flush=True)
    T = TYPES[dt]
    for R, residual, wide in ((1, True, False), (70 if K <= 4096 else 9, True, True), (41 if K <= 4096 else 5, False, False)):
        x, dy, dh = rows(R, K, T, K), rows(R, K, T, 1, 0.3), rows(R, K, T, 2, 0.3) if residual else None
        r = rows(R, K, T, 3) if residual else None
        w = rows(1, K, torch.float32 if wide else T, 4)[0]
        leaves = [t.cuda().requires_grad_() for t in ([x, w, r] if residual else [x, w])]
        out = norm.rms_norm(*leaves, eps=EPS)
        h = out[1].detach().cpu() if residual else x
        grads = torch.autograd.grad(out, leaves, [dy.cuda(), dh.cuda()] if residual else dy.cuda())
        h64, w64, dy64 = h.double(), w.double(), dy.double()
        dx, dw = gradient(dy64, dh.double() if residual else None, h64, w64, EPS)
        n = torch.sqrt(h64.square().mean(1, keepdim=True) + EPS)
        u = (h64 / n).abs()
        size = ((w64 * dy64).abs() + u * (w64 * dy64).abs().mul(u).mean(1, keepdim=True)) / n
        near(grads[0], dx, dx.abs() * half_step(T) + (size + (dh.double().abs() if residual else 0)) * FP32 + smallest(T), "dx")
        if residual:
            assert torch.equal(grads[0], grads[2])
        # at most 70 rows: under 128 additions in a row, and u's own error
        dw_size = (dy64.abs() * u).sum(0)
        near(grads[1], dw, dw.abs() * (0 if wide else half_step(T)) + dw_size * 2.0 ** -17 + smallest(T), "dw")
        assert grads[1].dtype == w.dtype


def test_many_rows():
    """More rows than the gradient has workgroups, each with several, and rows left over."""
    for K in (24, 300, 1500, 2500, 5000):
        print("many rows", K, flush=True)
        R = 2 * 1024 * (16 if K <= 128 else 4 if K <= 1024 else 1) + 5
        x, dy, w = rows(R, K, torch.bfloat16, 1), rows(R, K, torch.bfloat16, 2), rows(1, K, torch.bfloat16, 3)[0]
        leaves = [x.cuda().requires_grad_(), w.cuda().requires_grad_()]
        y = norm.rms_norm(*leaves, eps=EPS)
        dxg, dwg = torch.autograd.grad(y, leaves, dy.cuda())
        check_y(y.detach(), x, w)
        x64, dy64, w64 = x.double(), dy.double(), w.double()
        dx, dw = gradient(dy64, None, x64, w64, EPS)
        n = torch.sqrt(x64.square().mean(1, keepdim=True) + EPS)
        u = (x64 / n).abs()
        size = ((w64 * dy64).abs() + u * (w64 * dy64).abs().mul(u).mean(1, keepdim=True)) / n
        near(dxg, dx, dx.abs() * half_step(torch.bfloat16) + size * FP32, "dx")
        # fewer than 128 additions in a row again: 3 to 9 rows a thread, 16 groups, 64 parts, 16 waves
        near(dwg, dw, dw.abs() * half_step(torch.bfloat16) + (dy64.abs() * u).sum(0) * 2.0 ** -17, "dw")
        again = torch.autograd.grad(norm.rms_norm(*leaves, eps=EPS), leaves, dy.cuda())
        assert torch.equal(again[0], dxg) and torch.equal(again[1], dwg)


@pytest.mark.parametrize("K", [13, 96, 700, 1111, 4000])
def test_views(K):
    """Rows at any address and distance, rows that share memory, and what lies between rows."""
    print("views", K, flush=True)
    base = rows(9, K + 37, torch.float16, 1).cuda()
    w = rows(1, K + 1, torch.float16, 2).cuda()[0, 1:]
    x, r = base[:, 3:3 + K], base[:, 9:9 + K]
    y, h = norm.rms_norm(x, w, r, eps=EPS)
    assert torch.equal(h.cpu(), (x.float() + r.float()).half().cpu())
    check_y(y, h.cpu(), w.cpu())
    one = base[2:3, 5:5 + K].expand(6, K)
    y = norm.rms_norm(one, w, eps=EPS)
    check_y(y, one.cpu(), w.cpu())
    q, scale = i8.i8_quantize(x)
    check_rows(q, scale, x.cpu().double(), 0.0)
    # rows of outputs further apart than they are long: what lies between them stays
    import dense_tiled_gemm_02_amd as g
    out = torch.full((9, K + 11), 77, dtype=torch.int8, device="cuda")
    s = torch.empty(9, device="cuda")
    i8.gemm_i8_quantize(x.data_ptr(), g.GEMM_F16, 9, K, x.stride(0), out.data_ptr() + 1, K + 11, s.data_ptr(),
                        torch.cuda.current_stream().cuda_stream)
    assert torch.equal(out[:, 1:K + 1], q) and bool((out[:, 0] == 77).all()) and bool((out[:, K + 1:] == 77).all())
    # a broadcast gradient, as a sum's is
    leaf = x.detach().clone().requires_grad_()
    norm.rms_norm(leaf, w, eps=EPS).sum().backward()
    dx, _ = gradient(torch.ones(9, K, dtype=torch.float64), None, x.cpu().double(), w.cpu().double(), EPS)
    near(leaf.grad, dx, dx.abs() * half_step(torch.float16) + 2 * dx.abs().max() * 2.0 ** -14, "dx of a sum")


def test_values_at_the_ends():
    for dt in TYPES.values():
        big = torch.finfo(dt).max
        for K in (64, 1000, 3000, 20000):
            print("ends", dt, K, flush=True)
            x = rows(6, K, dt, 1)
            x[0] = 0
            x[1] = big
            x[2] = -big
            x[3, K // 2] = float("inf")
            x[4, 1] = float("nan")
            x[5] = smallest(dt)
            w = torch.ones(K, dtype=dt)
            y = norm.rms_norm(x.cuda(), w.cuda(), eps=EPS).cpu()
            fine = [0, 1, 2, 5]
            check_y(y[fine], x[fine], w)
            # inf / inf is NaN, finite / inf is 0
            assert bool(torch.isnan(y[3, K // 2])) and int(torch.isnan(y[3]).sum()) == 1
            assert float(y[3].nan_to_num(0.0).abs().max()) == 0.0 and bool(torch.isnan(y[4]).all())
            for q, scale in (i8.i8_quantize(x.cuda()), norm.rms_norm_i8(x.cuda(), w.cuda(), eps=EPS)):
                q, scale = q.cpu(), scale.cpu()
                assert bool((q[0] == 0).all()) and float(scale[0]) == 0.0
                assert bool((q[1] == 127).all()) and bool((q[2] == -127).all())
                assert bool((q[3:5] == 0).all()) and bool(torch.isnan(scale[3:5]).all())
                assert bool(torch.isfinite(scale[[1, 2, 5]]).all())
            # a row next to a bad one is its own
            assert torch.equal(norm.rms_norm(x[5:].cuda(), w.cuda(), eps=EPS).cpu(), y[5:])


def test_no_rows_and_no_values():
    w = torch.ones(8, dtype=torch.bfloat16, device="cuda").requires_grad_()
    x = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda").requires_grad_()
    y, h = norm.rms_norm(x, w, x)
    assert y.shape == (0, 8) and h.shape == (0, 8)
    dx, dw = torch.autograd.grad(y, (x, w), torch.empty_like(y))
    assert dx.shape == (0, 8) and torch.equal(dw, torch.zeros_like(w))
    empty = torch.empty(5, 0, dtype=torch.bfloat16, device="cuda")
    q, scale = i8.i8_quantize(empty)
    assert q.shape == (5, 0) and torch.equal(scale, torch.zeros(5, device="cuda"))
    q, scale, h = norm.rms_norm_i8(empty, w[:0].detach(), empty)
    assert q.shape == (5, 0) and torch.equal(scale, torch.zeros(5, device="cuda"))
    assert norm.rms_norm(empty, w[:0].detach()).shape == (5, 0)


def test_outputs_used_alone_and_inputs_that_need_no_gradient():
    x, r, w = rows(5, 96, torch.bfloat16, 1).cuda(), rows(5, 96, torch.bfloat16, 2).cuda(), rows(1, 96, torch.float32, 3)[0].cuda()
    d = rows(5, 96, torch.bfloat16, 4).cuda()
    leaf = r.clone().requires_grad_()
    y, h = norm.rms_norm(x, w, leaf, eps=EPS)
    assert torch.equal(torch.autograd.grad(h, leaf, d, retain_graph=True)[0], d)
    dx, _ = gradient(d.cpu().double(), None, h.detach().cpu().double(), w.cpu().double(), EPS)
    got = torch.autograd.grad(y, leaf, d)[0]
    assert float((got.cpu().double() - dx).norm()) <= 2.0 ** -7 * float(dx.norm())
    leaf = w.clone().requires_grad_()
    y = norm.rms_norm(x, leaf, eps=EPS)
    _, dw = gradient(d.cpu().double(), None, x.cpu().double(), w.cpu().double(), EPS)
    assert float((torch.autograd.grad(y, leaf, d)[0].cpu().double() - dw).norm()) <= 2.0 ** -16 * float(dw.norm())
    with torch.no_grad():
        assert not norm.rms_norm(x, leaf).requires_grad
    # one tensor as both addends: its gradient is the sum of both
    both = x.clone().requires_grad_()
    y, h = norm.rms_norm(both, w, both, eps=EPS)
    dx, _ = gradient(d.cpu().double(), None, h.detach().cpu().double(), w.cpu().double(), EPS)
    assert float((torch.autograd.grad(y, both, d)[0].cpu().double() - 2 * dx).norm()) <= 2.0 ** -7 * float(dx.norm()) * 2


def test_another_stream():
    s = torch.cuda.Stream()
    x, w = rows(2000, 1024, torch.float16, 1).cuda(), rows(1, 1024, torch.float16, 2)[0].cuda()
    want = norm.rms_norm(x, w), i8.i8_quantize(x), norm.rms_norm_i8(x, w)
    s.wait_stream(torch.cuda.current_stream())
    got = norm.rms_norm(x, w, stream=s), i8.i8_quantize(x, stream=s), norm.rms_norm_i8(x, w, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got[0], want[0])
    for a, b in zip(got[1] + got[2], want[1] + want[2]):
        assert torch.equal(a, b)


def test_captured_forward_and_backward():
    """Replayed with other values in the inputs, eager work in between."""
    R, K = 300, 1536
    static = [rows(R, K, torch.bfloat16, i).cuda().requires_grad_() for i in range(2)]
    w = rows(1, K, torch.bfloat16, 3)[0].cuda().requires_grad_()
    dy, dh = rows(R, K, torch.bfloat16, 4).cuda(), rows(R, K, torch.bfloat16, 5).cuda()

    def step():
        y, h = norm.rms_norm(static[0], w, static[1])
        q, s, h2 = norm.rms_norm_i8(static[0].detach(), w.detach(), static[1].detach())
        return [y.detach(), h.detach(), q, s, h2] + list(torch.autograd.grad((y, h), (static[0], w), (dy, dh)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(3):
        with torch.no_grad():
            static[0].copy_(rows(R, K, torch.bfloat16, 10 + i))
            static[1].copy_(rows(R, K, torch.bfloat16, 20 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_gradients_have_no_gradients():
    x, w = (rows(3, 64, torch.bfloat16, i).cuda().requires_grad_() for i in (1, 2))
    dx, = torch.autograd.grad(norm.rms_norm(x, w.detach()[0]).float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="not differentiable"):
        dx.float().sum().backward()


class Marked(torch.Tensor):
    """A tensor subclass: the calls that are remembered do not look at it."""


def test_other_tensor_types_and_calls_made_twice():
    x, r, w = rows(5, 200, torch.float16, 1).cuda(), rows(5, 200, torch.float16, 2).cuda(), rows(1, 200, torch.float32, 3)[0].cuda()
    first = norm.rms_norm(x, w, r), norm.rms_norm_i8(x, w, r), i8.i8_quantize(x)
    again = norm.rms_norm(x, torch.nn.Parameter(w), r), norm.rms_norm_i8(x, w, r), i8.i8_quantize(x)
    with torch.no_grad():
        marked = norm.rms_norm(x.as_subclass(Marked), w, r), norm.rms_norm_i8(x.as_subclass(Marked), w, r), \
            i8.i8_quantize(x.as_subclass(Marked))
    for a, b, c in zip(first, again, marked):
        for s, t, u in zip(a, b, c):
            assert torch.equal(s.detach(), t.detach()) and torch.equal(s, u.as_subclass(torch.Tensor))
    # what was not remembered is refused as before
    with pytest.raises(TypeError):
        norm.rms_norm(x, w.double(), r)
    with pytest.raises(Exception, match="eps"):
        norm.rms_norm(x, w, r, eps=0.0)


def test_many_rows_of_every_kind_of_row():
    """The shapes for more rows than a round, against the ones for few, bit by bit, and by value."""
    for K in (3000, 4096, 12001, 16384):
        print("many rows", K, flush=True)
        x, r = rows(700, K, torch.bfloat16, K).cuda(), rows(700, K, torch.bfloat16, K + 1).cuda()
        w = rows(1, K, torch.float32, 6)[0].cuda()
        q, scale = i8.i8_quantize(x)
        some = i8.i8_quantize(x[300:400])
        assert torch.equal(q[300:400], some[0]) and torch.equal(scale[300:400], some[1])
        y, h = norm.rms_norm(x, w, r, eps=EPS)
        check_y(y[-5:].cpu(), h[-5:].cpu(), w.cpu())
        assert torch.equal(h, (x.float() + r.float()).bfloat16())
        q, scale, h2 = norm.rms_norm_i8(x, w, r, eps=EPS)
        h64 = h[-5:].cpu().double()
        check_rows(q[-5:], scale[-5:], h64 * w.cpu().double() / torch.sqrt(h64.square().mean(1, keepdim=True) + EPS), FP32)
        assert torch.equal(h, h2)


def test_quotients_halfway_between_two_steps():
    """Values whose quotient is halfway, or next to it: rounded as an IEEE division's."""
    for dt in TYPES.values():
        x = torch.arange(-127, 128).to(dt).repeat(40, 1)
        x[:, 3] = 127
        for i in range(1, 40):
            x[i] = (x[0].float() * (0.5 + i / 64)).to(dt)
            x[i, 3] = 127
        x[10] = (x[0].float() - 0.5).to(dt)
        x[10, 3] = 127
        x[11] = x[10] * 2.0 ** -8
        q, scale = i8.i8_quantize(x.cuda())
        s = x.float().abs().amax(1) / 127
        assert torch.equal(scale.cpu(), s)
        assert torch.equal(q.cpu().float(), (x.float() / s[:, None]).round().clamp(-127, 127))
    # the smallest scales: their reciprocal is infinite, and quotients can pass 127
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    for i, v in enumerate((2.0 ** -133, 2.0 ** -126, 2.0 ** -101)):
        x[i] = torch.arange(-32, 32) / 32 * v
    q, scale = i8.i8_quantize(x.cuda())
    s = x.float().abs().amax(1) / 127
    assert torch.equal(scale.cpu(), s)
    want = torch.where(s[:, None] > 0, x.float() / s[:, None], torch.zeros(1)).round().clamp(-127, 127)
    assert torch.equal(q.cpu().float(), want)


@pytest.mark.parametrize("K", [(1 << 20) + 3, 1 << 24])
def test_long_rows(K):
    """In fp32 a sum of K values of one sign goes through K / 8192 + 8 + 26 additions in a row: a thread's
    chunks, a chunk's values, the threads and the waves."""
    fp32 = (K / 8192 + 40) * 2.0 ** -24
    x, dy = rows(2, K, torch.bfloat16, 1), rows(2, K, torch.bfloat16, 2)
    w = rows(1, K, torch.float32, 3)[0]
    dx_w = [t.cuda().requires_grad_() for t in (x, w)]
    y = norm.rms_norm(*dx_w, eps=EPS)
    u = half_step(torch.bfloat16)
    x64, w64, dy64 = x.double(), w.double(), dy.double()
    rstd = 1 / torch.sqrt(x64.square().mean(1, keepdim=True) + EPS)
    want = x64 * w64 * rstd
    near(y.detach(), want, want.abs() * (u + fp32) + smallest(torch.bfloat16), "y")
    q, scale = norm.rms_norm_i8(dx_w[0].detach(), dx_w[1].detach(), eps=EPS)
    most = want.abs().amax(1)
    near(scale, most / 127, most / 127 * (fp32 + 2.0 ** -20), "scale")
    near(q.cpu().double() * scale.cpu().double()[:, None], want, (most / 127 * 0.5)[:, None] + want.abs() * (fp32 + 2.0 ** -20), "q")
    dx, dw = torch.autograd.grad(y, dx_w, dy.cuda())
    g, v = dy64 * w64, x64 * rstd
    mean, off = (g * v).mean(1, keepdim=True), (g * v).abs().mean(1, keepdim=True)
    want = (g - v * mean) * rstd
    bound = want.abs() * (u + fp32) + ((g.abs() + v.abs() * mean.abs()) * (fp32 + 2.0 ** -21) + v.abs() * off * fp32) * rstd
    near(dx, want, bound + smallest(torch.bfloat16), "dx")
    near(dw, (dy64 * v).sum(0), (dy64 * v).abs().sum(0) * (fp32 + 2.0 ** -21), "dw")


def test_eps_counts_where_the_squares_overflow():
    """Values and eps near the largest: 1 / sqrt(mean + eps) of a mean past fp32's range."""
    x = torch.full((3, 40), 2.0 ** 64, dtype=torch.bfloat16)
    x[1] *= 2
    w = torch.ones(40, dtype=torch.bfloat16)
    y = norm.rms_norm(x.cuda(), w.cuda(), eps=3e38)
    want = x.double() / torch.sqrt(x.double().square().mean(1, keepdim=True) + 3e38)
    near(y, want, want * (half_step(torch.bfloat16) + FP32), "y")
