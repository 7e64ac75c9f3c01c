"""Which kernel a grouped product's plan takes on 256 CUs, at the sizes whose
tests on the GPU mean to run it (CPU)."""
import pytest

from test_grouped import plan, rows_problem


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("lens,N", [([4100], 4104), ([8200], 2200), ([7000, 3], 2312), ([3000, 3000, 3000, 200], 1928),
                                    ([2049, 2200, 2300], 2312), ([2500, 2500], 3336)], ids=str)
def test_two_sizes(lens, N, trans):
    assert "rows_mixed_kernel" in plan(rows_problem(E=len(lens), R=sum(lens) + 153, P=1000, Q=N, trans=trans)).describe()


def test_few_rows():
    for trans in (False, True):
        assert plan(rows_problem(E=8, R=16, P=1024, Q=512, trans=trans)).config.bm == 16
