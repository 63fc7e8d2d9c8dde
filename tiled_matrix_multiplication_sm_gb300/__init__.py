"""GB300-native tiled dense matrix multiplication, C = A x B.

The compute lives in ``libtgemm.so`` (CUDA for sm_103a, built from ``csrc/``
by :mod:`.build`); this package is its Python binding. See :mod:`.binding`
for the calls and :mod:`.mx4` for matrices in 4-bit floating point.
"""
from .binding import (  # noqa: F401
    TGEMM_TF32, TGEMM_BF16, TGEMM_TF32X3, TgemmError, load, library_path, gemm_f32, gemm_tc,
    gemm_f32_raw, gemm_tc_raw, device_status, status_string, matmul,
)

from .mx4 import (  # noqa: F401
    TGEMM_MXFP4, TGEMM_NVFP4, Mx4Matrix, mx4_tensor_scale, mx4_quantize, mx4_quantize_both,
    mx4_dequantize, mx4_pack, gemm_mx4, gemm_w4,
)

__all__ = ["TGEMM_TF32", "TGEMM_BF16", "TGEMM_TF32X3", "TgemmError", "load", "library_path",
           "gemm_f32", "gemm_tc", "gemm_f32_raw", "gemm_tc_raw",
           "device_status", "status_string", "matmul",
           "TGEMM_MXFP4", "TGEMM_NVFP4", "Mx4Matrix", "mx4_tensor_scale", "mx4_quantize",
           "mx4_quantize_both", "mx4_dequantize", "mx4_pack", "gemm_mx4", "gemm_w4"]
