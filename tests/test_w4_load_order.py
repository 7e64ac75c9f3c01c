"""The order of loads that the 4-bit kernels' waits count on, read from the
library built here (CPU).

A step of the main loop waits for its X, in LDS, by the number of loads that
were issued after it: X's loads have to go out before W's.  So the first 16-byte
load after each wait that leaves loads in flight is one to LDS, in every
variant."""
import os
import re
import struct
import subprocess

import pytest

import dense_tiled_gemm_02_amd as g
from dense_tiled_gemm_02_amd import build

OBJDUMP = os.path.join(os.path.dirname(os.path.dirname(build.HIPCC)), "llvm", "bin", "llvm-objdump")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(path):
    """The gfx950 ELF images in a library's offload bundles."""
    data = open(path, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        n, = struct.unpack_from("<Q", data, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(n):
            off, size, length = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + length]
            p += 24 + length
            if name.endswith(b"gfx950"):
                yield data[at + off:at + off + size]
        at = data.find(MAGIC, p)


def kernels(tmp_path):
    """{name: lines of assembly} of the 4-bit kernels."""
    found = {}
    for image in code_objects(g.LIB_PATH):
        if b"gemm_w4_kernel" not in image:
            continue
        path = tmp_path / "code.o"
        path.write_bytes(image)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--mcpu=gfx950", str(path)], check=True,
                              capture_output=True, text=True).stdout
        for part in re.split(r"^[0-9a-f]+ <", text, flags=re.M)[1:]:
            name, _, body = part.partition(">:")
            if "gemm_w4_kernel" in name:
                found[name] = [l.strip() for l in body.splitlines()]
    return found


def misplaced(lines):
    """(loads checked, loads out of order) of one kernel."""
    checked, wrong, in_flight = 0, [], False
    for l in lines:
        wait = re.search(r"vmcnt\((\d+)\)", l)
        if wait:
            in_flight = in_flight or int(wait.group(1)) > 0
        elif l.startswith(("global_load_lds", "global_load_dwordx4")):
            checked += in_flight
            if in_flight and not l.startswith("global_load_lds"):
                wrong.append(l)
            in_flight = False
    return checked, wrong


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_x_goes_out_before_w(tmp_path):
    found = kernels(tmp_path)
    assert len(found) >= 100
    for name, lines in found.items():
        checked, wrong = misplaced(lines)
        assert checked > 0 and not wrong, (name, checked, wrong[:3])


def test_the_reading_sees_a_swap():
    right = ["s_waitcnt vmcnt(6)", "v_mfma_f32_16x16x32_f16 a", "global_load_lds_dwordx4 v[0:1], off",
             "global_load_dwordx4 v[2:5], v[0:1], off", "s_waitcnt vmcnt(0)", "global_load_dwordx4 v[2:5], v[0:1], off"]
    assert misplaced(right) == (1, [])
    assert misplaced([right[0], right[3], right[2]]) == (1, [right[3]])
