"""The norm's weight gradient over so many rows that every thread takes some 2048 of
them (GPU).

Every term is the same number c, whose last bits a running fp32 sum past 1024 loses
each time: 2^-15 of the whole, 490 x 2^-24.  The sum's additions in a row: 128 rows of a
thread, 15 threads side by side, 63 of 64 workgroups' parts, 15 of 16 waves; and, where
there are more than 1024 parts (up to 17 sums of 1024 here), one of 2 a wave and 15 of
the waves again: 237, and the product's and the output's rounding.  Each is off by at
most 2^-24 of a sum that is no larger than the whole."""
import pytest
import torch

from dense_tiled_gemm_02_amd import norm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


# of K: about how many rows a launch has under way, as many threads to each column
@pytest.mark.parametrize("K, at_once", [(72, 16384), (700, 3000), (2000, 1024), (4000, 512), (8200, 256), (16400, 256)])
def test_equal_terms(K, at_once):
    print("equal terms", K, flush=True)
    R = 2048 * at_once + 5
    one = torch.ones(1, K, dtype=torch.bfloat16, device="cuda").expand(R, K)   # rows share memory
    c = torch.tensor(1 + 0.49 * 2.0 ** -13, dtype=torch.float32)
    rstd = c.cuda().expand(R).contiguous()
    weight = torch.ones(K, device="cuda")
    dx, dw = norm.rms_norm_grad(one, one, weight, rstd)
    want = R * c.double()
    assert float((dw.cpu().double() - want).abs().max() / want) <= 239 * 2.0 ** -24
    # dx of equal terms: g - u mean(g u), which is 1 - c^2, times c; four roundings of numbers next to 1
    want = float((1 - c.double() ** 2) * c.double())
    for rows in (dx[:3], dx[-3:]):
        assert float((rows.double() - want).abs().max()) <= abs(want) * 2.0 ** -8 + 4 * K.bit_length() * 2.0 ** -24
    again = norm.rms_norm_grad(one, one, weight, rstd)[1]
    assert torch.equal(again, dw)


def test_random_terms_of_one_sign():
    K, R = 40, 3 * (1 << 22) + 7   # 768 rows a thread
    gen = torch.Generator(device="cuda").manual_seed(1)
    h, dy = (torch.rand(R, K, generator=gen, device="cuda").add_(0.5).half() for _ in range(2))
    rstd = torch.rand(R, generator=gen, device="cuda") + 0.5
    want = torch.zeros(K, dtype=torch.float64, device="cuda")
    for i in range(0, R, 1 << 19):
        at = slice(i, i + (1 << 19))
        want += (dy[at].double() * h[at].double() * rstd[at, None].double()).sum(0)
    dw = norm.rms_norm_grad(dy, h, torch.ones(K, device="cuda"), rstd)[1]
    # and u = h rstd is rounded before its product
    assert float(((dw.double() - want).abs() / want).max()) <= 240 * 2.0 ** -24
