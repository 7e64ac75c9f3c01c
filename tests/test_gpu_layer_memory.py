"""Out of memory is torch's own error, from remembered calls and checked ones, and an
error that a hook raises is the hook's (GPU)."""
import contextlib

import pytest
import torch

from dense_tiled_gemm_02_amd import i8, norm, router

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def a_gigabyte():
    """This process may hold that much and no more."""
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction((1 << 30) / torch.cuda.get_device_properties(0).total_memory)
    try:
        yield
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
        torch.cuda.empty_cache()


def calls():
    """Outputs of 2 GiB and more, from rows that share memory."""
    K, R = 1 << 14, 1 << 17
    row = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    w, s = torch.ones(K, device="cuda"), torch.ones(1 << 15, device="cuda")
    many, leaf = row.expand(R, K), row.clone().requires_grad_().expand(R, K)
    x = torch.zeros(1, 64, dtype=torch.int8, device="cuda").expand(1 << 15, 64)
    logits = torch.zeros(1, 64, device="cuda").expand(1 << 23, 64)
    return [lambda: norm.rms_norm(many, w), lambda: norm.rms_norm(leaf, w), lambda: norm.rms_norm_i8(many, w),
            lambda: i8.i8_quantize(many), lambda: router.route(logits, 64), lambda: i8.i8_matmul(x, s, x, s)]


@pytest.mark.parametrize("which", range(6))
@pytest.mark.parametrize("remembered", [False, True])
def test_out_of_memory_is_torchs_error(which, remembered):
    call = calls()[which]
    if remembered:
        call()
    else:
        from dense_tiled_gemm_02_amd import grouped
        grouped._native().forget()
    with a_gigabyte():
        with pytest.raises(torch.OutOfMemoryError):
            call()
    out = call()   # what comes after it runs
    assert out is not None


class Full(ValueError):
    pass


@pytest.mark.parametrize("remembered", [False, True])
def test_an_error_of_a_hook_is_the_hooks(remembered):
    def full(t):
        raise Full("no room")

    x, w = torch.randn(3, 64, device="cuda").half().requires_grad_(), torch.ones(64, device="cuda")
    calls = (lambda: norm.rms_norm(x, w), lambda: router.route(x, 2))
    for call in calls:
        if remembered:
            call()
        with torch.autograd.graph.saved_tensors_hooks(full, lambda t: t):
            with pytest.raises(Full, match="no room"):
                call()
        call()
