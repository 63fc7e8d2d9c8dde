"""4-bit floating-point matrices: the binding of ``include/tgemm_mx4.h``.

:class:`Mx4Matrix` holds a matrix in 4 bits (E2M1 codes with block scales, in
the layout the tensor core reads); :func:`mx4_quantize` makes one from a BF16
or FP32 tensor, :func:`mx4_pack` from row-major codes and scales. Products:
:func:`gemm_mx4` (both operands in 4 bits) and :func:`gemm_w4` (BF16
activations with 4-bit weights). Argument marshalling only, as in
:mod:`.binding`; every call is asynchronous on ``stream`` (default: the
current one), and what a call allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import binding
from .binding import TGEMM_OK, TgemmError, _stream_handle

TGEMM_MXFP4 = 1
TGEMM_NVFP4 = 2
TGEMM_MX4_SET_G = 1
TGEMM_TYPE_F32 = 0
TGEMM_TYPE_BF16 = 1

_FORMATS = {"mxfp4": TGEMM_MXFP4, "nvfp4": TGEMM_NVFP4}
_BLOCK = {"mxfp4": 32, "nvfp4": 16}
_TYPES = {torch.float32: TGEMM_TYPE_F32, torch.bfloat16: TGEMM_TYPE_BF16}

_INT, _LONG, _FLT, _VP = ctypes.c_int, ctypes.c_long, ctypes.c_float, ctypes.c_void_p
_OUT = [_VP, _LONG, _INT, _FLT, _FLT, _VP, _VP]          # C, ldc, type, alpha, beta, bias, stream
_SIGNATURES = {
    "gemm_mx4_codes_pitch": (ctypes.c_longlong, [_INT]),
    "gemm_mx4_scales_bytes": (ctypes.c_longlong, [_INT, _INT, _INT]),
    "gemm_mx4_tensor_scale": (_INT, [_INT, _INT, _VP, _LONG, _INT, _VP, _VP]),
    "gemm_mx4_quantize": (_INT, [_INT, _INT, _VP, _LONG, _INT, _INT, _VP, _INT, _VP, _VP, _VP, _VP, _VP]),
    "gemm_mx4_dequantize": (_INT, [_INT, _INT, _VP, _VP, _INT, _VP, _VP, _LONG, _INT, _VP]),
    "gemm_mx4_pack": (_INT, [_INT, _INT, _INT, _VP, _LONG, _VP, _LONG, _VP, _VP, _VP]),
    "gemm_mx4": (_INT, [_INT, _INT, _INT, _VP, _VP, _VP, _VP, _VP, _VP, _INT] + _OUT),
    "gemm_w4": (_INT, [_INT, _INT, _INT, _VP, _LONG, _VP, _VP, _VP, _INT] + _OUT),
}

_lib = None


def load() -> ctypes.CDLL:
    """libtgemm.so with these entry points declared."""
    global _lib
    if _lib is None:
        lib = binding.load()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _call(name: str, device: torch.device, stream: Optional[torch.cuda.Stream], *args) -> None:
    """Run entry point ``name`` with ``args`` and the stream on ``device``;
    switches devices only when another one is current."""
    fn = getattr(_lib or load(), name)
    index = device.index
    if index is None or index == torch.cuda.current_device():
        status = fn(*args, _stream_handle(stream, index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _stream_handle(stream, index))
    if status != TGEMM_OK:
        raise TgemmError(status, name)


def _format(fmt: str) -> int:
    if fmt not in _FORMATS:
        raise ValueError(f"unknown 4-bit format {fmt!r}; have {sorted(_FORMATS)}")
    return _FORMATS[fmt]


def _type(dtype: torch.dtype, name: str) -> int:
    if dtype not in _TYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")
    return _TYPES[dtype]


def _empty(stream: Optional[torch.cuda.Stream], *size, dtype, device) -> torch.Tensor:
    """torch.empty, of memory that belongs to ``stream`` (default: the current one)."""
    if stream is None:
        return torch.empty(size, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=dtype, device=device)


def _check_scale(g: Optional[torch.Tensor], fmt: str, device: torch.device) -> int:
    """The pointer of a tensor scale (0: none)."""
    if g is None:
        return 0
    if fmt != "nvfp4":
        raise ValueError("only nvfp4 matrices have a tensor scale")
    if not isinstance(g, torch.Tensor) or g.dtype != torch.float32 or g.numel() != 1:
        raise TypeError("tensor_scale must be a float32 tensor of one element")
    if g.device != device:
        raise ValueError(f"tensor_scale is on {g.device}, the matrix on {device}")
    return g.data_ptr()


def _sizes(rows: int, cols: int, fmt: str) -> Tuple[int, int]:
    """Bytes of the codes and of the scales of a matrix: rows times
    gemm_mx4_codes_pitch, and gemm_mx4_scales_bytes."""
    _format(fmt)
    if rows < 0 or cols < 0:
        raise ValueError(f"a 4-bit matrix cannot be {rows} x {cols}")
    return (rows * ((cols + 31) // 32 * 16),
            (rows + 127) // 128 * ((cols + 255) // 256) * (32768 // _BLOCK[fmt]))


class Mx4Matrix:
    """A ``rows`` x ``cols`` matrix in 4 bits, quantised along its columns
    (the axis a product sums over): ``codes``, ``scales`` (uint8, in the
    library's layout) and, for nvfp4, ``tensor_scale`` (one float32)."""

    __slots__ = ("fmt", "rows", "cols", "shape", "device", "tensor_scale", "_held", "_codes", "_scales", "_g")

    def __init__(self, fmt: str, rows: int, cols: int, codes: torch.Tensor, scales: torch.Tensor,
                 tensor_scale: Optional[torch.Tensor] = None):
        for t, size, name in zip((codes, scales), _sizes(rows, cols, fmt), ("codes", "scales")):
            if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous() or t.numel() < size:
                raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor of {size} bytes")
        if codes.device != scales.device:
            raise ValueError("codes and scales are on different devices")
        self._set(fmt, rows, cols, (codes, scales), codes.data_ptr(), scales.data_ptr(), codes.device,
                  tensor_scale, _check_scale(tensor_scale, fmt, codes.device))

    def _set(self, fmt, rows, cols, held, codes, scales, device, tensor_scale, g):
        self.fmt, self.rows, self.cols, self.shape, self.device = fmt, rows, cols, (rows, cols), device
        self._held, self._codes, self._scales = held, codes, scales
        self.tensor_scale, self._g = tensor_scale, g

    @classmethod
    def _empty(cls, fmt, rows, cols, device, tensor_scale, g, stream) -> "Mx4Matrix":
        """An unwritten matrix, codes and scales in one allocation."""
        n, m = _sizes(rows, cols, fmt)
        data = _empty(stream, n + m, dtype=torch.uint8, device=device)
        at = data.data_ptr()
        self = cls.__new__(cls)
        self._set(fmt, rows, cols, (data, n), at, at + n, device, tensor_scale, g)
        return self

    @property
    def codes(self) -> torch.Tensor:
        data, n = self._held
        return data[:n] if isinstance(n, int) else data

    @property
    def scales(self) -> torch.Tensor:
        data, n = self._held
        return data[n:] if isinstance(n, int) else n

    def __repr__(self) -> str:
        return f"Mx4Matrix({self.fmt}, {self.rows} x {self.cols}, {self.device})"


def _check_mx4(m, name: str) -> None:
    if not isinstance(m, Mx4Matrix):
        raise TypeError(f"{name} must be an Mx4Matrix, got {type(m).__name__}")


def _check_matrix(x: torch.Tensor, name: str, dtype: torch.dtype) -> int:
    """The leading dimension of a row-major matrix whose rows do not overlap
    (an expanded one's do)."""
    ld = binding._check_matrix(x, name, dtype)
    if x.shape[0] > 1 and x.stride(0) < x.shape[1]:
        raise ValueError(f"{name}'s rows overlap: stride {x.stride(0)} for {x.shape[1]} columns")
    return ld


def _check_values(X: torch.Tensor, name: str) -> Tuple[int, int]:
    """(leading dimension, TGEMM_TYPE_*) of a float32 or bfloat16 matrix."""
    if not isinstance(X, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return _check_matrix(X, name, X.dtype), _type(X.dtype, name)


def mx4_tensor_scale(X: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The nvfp4 scale of X: the smallest power of two g with 2688 g >= |X|
    (one float32 on X's device; infinities and NaN are left out)."""
    ldx, kind = _check_values(X, "X")
    g = _empty(stream, 1, dtype=torch.float32, device=X.device)
    _call("gemm_mx4_tensor_scale", X.device, stream, X.shape[0], X.shape[1], X.data_ptr(), ldx, kind, g.data_ptr())
    return g


def _quantize(X, fmt, tensor_scale, stream, rows: bool, trans: bool):
    code = _format(fmt)
    ldx, kind = _check_values(X, "X")
    R, C = X.shape
    device = X.device
    set_g = fmt == "nvfp4" and tensor_scale is None
    if set_g:
        tensor_scale = _empty(stream, 1, dtype=torch.float32, device=device)
    g = _check_scale(tensor_scale, fmt, device)
    q = Mx4Matrix._empty(fmt, R, C, device, tensor_scale, g, stream) if rows else None
    t = Mx4Matrix._empty(fmt, C, R, device, tensor_scale, g, stream) if trans else None
    _call("gemm_mx4_quantize", device, stream, R, C, X.data_ptr(), ldx, kind, code, g,
          TGEMM_MX4_SET_G if set_g else 0, q._codes if rows else 0, q._scales if rows else 0,
          t._codes if trans else 0, t._scales if trans else 0)
    return q, t


def mx4_quantize(X: torch.Tensor, fmt: str = "mxfp4", trans: bool = False,
                 tensor_scale: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> Mx4Matrix:
    """X (float32 or bfloat16, row-major) in 4 bits along its rows, or with
    ``trans`` its transpose, in 4 bits along X's columns. ``fmt`` is "mxfp4"
    or "nvfp4"; nvfp4 takes ``tensor_scale`` (for one kept from an earlier
    step) or computes it from X."""
    return _quantize(X, fmt, tensor_scale, stream, not trans, trans)[1 if trans else 0]


def mx4_quantize_both(X: torch.Tensor, fmt: str = "mxfp4",
                      tensor_scale: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> Tuple[Mx4Matrix, Mx4Matrix]:
    """(X, its transpose) in 4 bits, X read once: what the forward and
    backward products of a layer take of the same matrix."""
    return _quantize(X, fmt, tensor_scale, stream, True, True)


def mx4_dequantize(Q: Mx4Matrix, dtype: torch.dtype = torch.float32,
                   out: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The values Q stands for, as float32 or bfloat16."""
    _check_mx4(Q, "Q")
    if out is None:
        _type(dtype, "dtype")
        out = _empty(stream, Q.rows, Q.cols, dtype=dtype, device=Q.device)
    elif tuple(out.shape) != Q.shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {Q.shape}")
    elif out.device != Q.device:
        raise ValueError(f"out is on {out.device}, the matrix on {Q.device}")
    ldx, kind = _check_values(out, "out")
    _call("gemm_mx4_dequantize", Q.device, stream, Q.rows, Q.cols, Q._codes, Q._scales, _FORMATS[Q.fmt], Q._g,
          out.data_ptr(), ldx, kind)
    return out


def mx4_pack(codes: torch.Tensor, scales: torch.Tensor, fmt: str = "mxfp4",
             cols: Optional[int] = None, tensor_scale: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> Mx4Matrix:
    """A matrix that comes in 4 bits, row-major, as a checkpoint holds it:
    ``codes`` uint8 (rows, ceil(cols / 2)), the lower column in the low half;
    ``scales`` uint8 (rows, ceil(cols / block)), E8M0 or E4M3 bytes. ``cols``
    defaults to twice the codes' width. ``tensor_scale`` is kept, not copied."""
    code = _format(fmt)
    if codes.numel() == 0:                 # an empty tensor's strides say nothing
        codes, scales = codes.new_empty(codes.shape), scales.new_empty(scales.shape)
    ldc = _check_matrix(codes, "codes", torch.uint8)
    lds = _check_matrix(scales, "scales", torch.uint8)
    rows = codes.shape[0]
    cols = 2 * codes.shape[1] if cols is None else int(cols)
    blocks = -(-cols // _BLOCK[fmt])
    if cols < 0 or codes.shape[1] != (cols + 1) // 2:
        raise ValueError(f"codes have {codes.shape[1]} bytes a row, {cols} columns need {(cols + 1) // 2}")
    if tuple(scales.shape) != (rows, blocks):
        raise ValueError(f"scales have shape {tuple(scales.shape)}, expected {(rows, blocks)}")
    if scales.device != codes.device:
        raise ValueError("codes and scales are on different devices")
    g = _check_scale(tensor_scale, fmt, codes.device)
    q = Mx4Matrix._empty(fmt, rows, cols, codes.device, tensor_scale, g, stream)
    _call("gemm_mx4_pack", codes.device, stream, rows, cols, code, codes.data_ptr(), ldc, scales.data_ptr(), lds,
          q._codes, q._scales)
    return q


def _output(out, M, N, out_dtype, device, beta, bias, stream):
    """(C, ldc, type, bias pointer) of a product."""
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs out, the C it scales")
        ldc, kind = max(N, 1), _type(out_dtype, "out_dtype")
        out = _empty(stream, M, N, dtype=out_dtype, device=device)
    else:
        ldc, kind = _check_values(out, "out")
        if tuple(out.shape) != (M, N):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(M, N)}")
        if out.device != device:
            raise ValueError(f"out is on {out.device}, the operands on {device}")
    if bias is None:
        return out, ldc, kind, 0
    if not isinstance(bias, torch.Tensor) or bias.dtype != torch.float32 or tuple(bias.shape) != (N,):
        raise ValueError(f"bias must be a float32 tensor of {N} elements")
    if bias.device != device or (N > 1 and bias.stride(0) != 1):
        raise ValueError("bias must be contiguous and on the operands' device")
    return out, ldc, kind, bias.data_ptr()


def gemm_mx4(A: Mx4Matrix, B: Mx4Matrix, out_dtype: torch.dtype = torch.float32,
             alpha: float = 1.0, beta: float = 0.0, bias: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """C = alpha * A @ B.T + beta * C + bias for A (M x K) and B (N x K), both
    in the same 4-bit format; C float32 or bfloat16 (``out``, or new)."""
    _check_mx4(A, "A")
    _check_mx4(B, "B")
    if A.cols != B.cols:
        raise ValueError(f"inner dimensions differ: {A.shape} x {B.shape} transposed")
    if A.fmt != B.fmt:
        raise ValueError(f"A is {A.fmt}, B is {B.fmt}")
    if A.device != B.device:
        raise ValueError(f"A is on {A.device}, B on {B.device}")
    C, ldc, kind, bias_ptr = _output(out, A.rows, B.rows, out_dtype, A.device, beta, bias, stream)
    _call("gemm_mx4", A.device, stream, A.rows, B.rows, A.cols, A._codes, A._scales, A._g, B._codes, B._scales,
          B._g, _FORMATS[A.fmt], C.data_ptr(), ldc, kind, alpha, beta, bias_ptr)
    return C


def gemm_w4(A: torch.Tensor, W: Mx4Matrix, out_dtype: torch.dtype = torch.float32,
            alpha: float = 1.0, beta: float = 0.0, bias: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """C = alpha * A @ W.T + beta * C + bias for bfloat16 A (M x K, row-major)
    and W (N x K) in 4 bits; C float32 or bfloat16 (``out``, or new)."""
    _check_mx4(W, "W")
    lda = _check_matrix(A, "A", torch.bfloat16)
    if A.shape[1] != W.cols:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} x {W.shape} transposed")
    if A.device != W.device:
        raise ValueError(f"A is on {A.device}, W on {W.device}")
    C, ldc, kind, bias_ptr = _output(out, A.shape[0], W.rows, out_dtype, A.device, beta, bias, stream)
    _call("gemm_w4", A.device, stream, A.shape[0], W.rows, W.cols, A.data_ptr(), lda, W._codes, W._scales, W._g,
          _FORMATS[W.fmt], C.data_ptr(), ldc, kind, alpha, beta, bias_ptr)
    return C
