"""The launch that a 4-bit plan describes (CPU)."""
import pytest

from dense_tiled_gemm_02_amd import w4
from test_abi import fake_gfx950
from test_grouped import w4_problem


@pytest.mark.parametrize("M,experts,rows", [(3, 0, 1), (3, 16, 3), (1, 41, 1), (16, 16, 16), (64, 100, 64), (65, 100, 100),
                                            (40, 16, 16)])
def test_workgroups_follow_the_rows_or_the_experts(M, experts, rows):
    text = w4.gemm_w4_plan_create_for(w4_problem(M=M, experts=experts), fake_gfx950()).describe()
    columns = int(text.split("columns=")[1].split()[0])
    assert text.endswith("grid=%dx%d" % (-(-256 // columns), rows))
