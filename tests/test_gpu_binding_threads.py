"""Remembered calls let other Python threads run while they allocate and launch,
and keep their plan while they do.  A C function that only waits stands in for
the library's launch."""
import ctypes
import gc
import threading
import time
import weakref

import pytest
import torch

import dense_tiled_gemm_02_amd as g
from dense_tiled_gemm_02_amd import grouped

pytestmark = pytest.mark.gpu
WAIT_US = 300000


class Owner:
    pass


def test_other_threads_run_and_the_plan_stays():
    binding = g.binding()
    x = torch.zeros(3, 5, dtype=torch.float16, device="cuda")
    owner = Owner()
    alive = weakref.ref(owner)
    usleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value   # its argument is the plan, its result 0
    tensors = (x, None, None, None, None)
    binding.remember(grouped.W4, owner, WAIT_US, usleep, 0, (2, 7), torch.float16, 12345, tensors)
    del owner
    seen = {}

    def caller():
        start = time.perf_counter()
        out = binding.call(grouped.W4, 12345, *tensors)
        seen["span"] = (start, time.perf_counter())
        seen["out"] = (tuple(out.shape), out.dtype)

    ticks, kept = [], []
    thread = threading.Thread(target=caller)
    thread.start()
    while thread.is_alive():
        time.sleep(0.002)
        ticks.append(time.perf_counter())
        if len(ticks) == 10:
            binding.forget()   # the table's reference goes
            gc.collect()
        if len(ticks) == 20:
            kept.append(alive() is not None)
    thread.join()
    start, end = seen["span"]
    assert end - start >= 0.9 * WAIT_US * 1e-6
    assert sum(start < t < end for t in ticks) >= 20
    assert kept == [True] and seen["out"] == ((2, 7), torch.float16)
    gc.collect()
    assert alive() is None
    assert binding.call(grouped.W4, 12345, *tensors) is None   # forgotten
