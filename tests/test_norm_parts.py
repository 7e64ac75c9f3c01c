"""The workspace of the norm's weight gradient: one row of fp32 sums for each
workgroup, none of whose threads adds more than 128 rows in a row (CPU)."""
import pytest

from dense_tiled_gemm_02_amd import norm
from test_norm import problem

# of K: the rows that a workgroup takes side by side, and the workgroups of a launch
SHAPES = [(1, 16, 1024), (128, 16, 1024), (129, 4, 768), (1024, 4, 768), (1025, 1, 1024), (2048, 1, 1024), (4096, 1, 512),
          (4097, 1, 256), (16384, 1, 256), (16385, 1, 256), (40000, 1, 256)]


def parts(R, K):
    n = norm.gemm_rms_norm_grad_workspace(problem(R, K))
    assert n % (4 * K) == 0
    return n // (4 * K)


@pytest.mark.parametrize("K, side, most", SHAPES)
def test_rows_of_a_thread(K, side, most):
    launch = 128 * side * most
    for R in (1, side, side + 1, 1000, 8192, launch - 1, launch, launch + 1, launch + side, 3 * launch - 7, 40 * launch + 12345,
              (1 << 31) - 4096):
        n = parts(R, K)
        whole, rest = divmod(R, launch)
        groups = -(-rest // side)
        # whole launches have all their workgroups, the last one no more, and no idle ones
        assert n - whole * most <= min(most, groups)
        assert rest == 0 or -(-groups // (n - whole * most)) <= 128
        # 128 rows of a thread and more than a row each, so little memory beside dx (2 bytes a value)
        assert R < launch or n * 4 * K <= R * K * 2 // 8
    assert parts(0, K) == 0


@pytest.mark.parametrize("K, side, most", SHAPES)
def test_ordinary_sizes_have_one_launch(K, side, most):
    """Four rows of a thread and more, down to 256 workgroups, up to `most`."""
    for R in (1, 77, 1024, 4096, 16384):
        need = -(-R // side)
        assert parts(R, K) == min(need, max(256, min(most, (need + 3) // 4)))
