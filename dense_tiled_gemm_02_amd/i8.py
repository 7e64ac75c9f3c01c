"""Rows in 8 bits with a scale for each (include/gemm.h).

    q, scale = i8_quantize(X)             # X: R x K, float16 or bfloat16

Argument marshalling only: the work runs in libgemm.so's HIP kernels.
"""
import torch

from . import GEMM_BF16, GEMM_F16, _check, lib
from .grouped import _need_gpu, _on_stream, _raw_stream
from .norm import _rows_arg

_CODES = {torch.float16: GEMM_F16, torch.bfloat16: GEMM_BF16}


def gemm_i8_quantize(x, dtype, R, K, sx, q, sq, scale, stream=None):
    """Device addresses (integers or None) and a hipStream_t (or None)."""
    _check(lib().gemm_i8_quantize(x, dtype, R, K, sx, q, sq, scale, stream))


# ---------------------------------------------------------------- torch convenience

def i8_quantize(X, stream=None):
    """(q, scale): each row of X (R x K, float16 or bfloat16, unit stride along the
    rows) as int8 steps of its own float32 scale, its largest magnitude / 127, so
    that X[i] is about q[i] scale[i]: activations with a scale per token, or a
    weight (N x K) with one per channel.  A row of zeros has the scale 0, a row
    with an infinity or a NaN the scale NaN.  No gradients.  Asynchronous on
    `stream` (default: torch's current stream)."""
    _rows_arg("X", X)
    _need_gpu(X.device, ("X", X))

    def call():
        R, K = X.shape
        q = torch.empty((R, K), dtype=torch.int8, device=X.device)
        scale = torch.empty(R, dtype=torch.float32, device=X.device)
        gemm_i8_quantize(X.data_ptr(), _CODES[X.dtype], R, K, X.stride(0), q.data_ptr(), K, scale.data_ptr(),
                         _raw_stream(X.device.index))
        return q, scale
    return _on_stream(call, X.device, stream, (X,))
