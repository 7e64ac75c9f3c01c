"""Resource gate of the kernels around the products: norm, 8-bit rows, int8 products
with scales, routing (CPU).  Scratch and vector spills of every kernel in the library
are test_resources.py's."""
import re

from test_resources import _demangle, report   # noqa: F401 (a fixture)

# kernels of each family, and the scalar registers that one may keep in a vector register's
# lanes: few outside the rows of four chunks, whose addresses are that many
FAMILIES = {"rows_kernel": (72, 28), "norm_grad_kernel": (16, 4), "norm_weight_grad_kernel": (6, 0), "route_kernel": (66, 4),
            "route_grad_kernel": (21, 0), "gemm_i8s_kernel": (18, 0), "gemm_i8s_mixed_kernel": (3, 0), "i8_few_kernel": (18, 0),
            "i8_any_kernel": (9, 0)}


def kernels(report):
    names = _demangle(list(report["kernels"]))
    for k, v in report["kernels"].items():
        found = re.search(r"(\w+)<([^>]*)>\(", names[k])
        if found and found.group(1) in FAMILIES:
            yield found.group(1), found.group(2).split(", "), v


def test_every_kernel_is_in_the_report(report):
    count = dict.fromkeys(FAMILIES, 0)
    for family, _, _ in kernels(report):
        count[family] += 1
    assert count == {family: n for family, (n, _) in FAMILIES.items()}


def test_scalar_spills(report):
    bad = [(family, args, v["SGPRs Spill"]) for family, args, v in kernels(report) if v["SGPRs Spill"] > FAMILIES[family][1]]
    assert not bad
    # of the rows' kernels, those of four chunks alone
    bad = [(args, v["SGPRs Spill"]) for family, args, v in kernels(report)
           if family == "rows_kernel" and args[2] != "4" and v["SGPRs Spill"] > 0]
    assert not bad


def test_waves_to_a_simd(report):
    """What the measured shapes were chosen with: several rows to a CU, one of which
    waits while another is worked on."""
    for family, args, v in kernels(report):
        if family == "rows_kernel" and args[2] in ("1", "2"):
            assert v["Occupancy"] >= 7, (family, args, v)
        elif family in ("rows_kernel", "norm_grad_kernel", "route_kernel"):
            assert v["Occupancy"] >= 4, (family, args, v)
        elif family in ("gemm_i8s_kernel", "gemm_i8s_mixed_kernel"):
            assert v["Occupancy"] >= 2, (family, args, v)
