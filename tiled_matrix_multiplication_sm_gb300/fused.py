"""Products with what follows them in a model's layers: the binding of
``include/tgemm_fused.h``.

:func:`gemm_act` is a layer's product with its bias, activation (gated or not)
and residual, :func:`gemm_act_grad` the backward pass through an activation;
:func:`gemm_ce` is the softmax cross entropy of a head over its vocabulary,
without keeping the logits, :func:`gemm_ce_grad` its gradients. Matrices are
bfloat16 and row-major (any leading dimension), results bfloat16 or float32.
Argument marshalling only, as in :mod:`.binding`; every call is asynchronous on
``stream`` (default: the current one), and what a call allocates belongs to
that stream. Results have no autograd history, whatever ``requires_grad`` their
operands have: the gradients are calls of their own, for a
``torch.autograd.Function`` to make (``examples/fused_ffn.py`` has a layer's and a head's).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple, Union

import torch

from . import binding
from .binding import TGEMM_OK, TGEMM_TRANS_A, TGEMM_TRANS_B, TgemmError, _stream_handle
from .mx4 import TGEMM_TYPE_BF16, _TYPES, _check_matrix, _check_values, _empty, _type

TGEMM_GATED = 4

_ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_INT, _LONG, _FLT, _VP = ctypes.c_int, ctypes.c_long, ctypes.c_float, ctypes.c_void_p
_SIZES = [_INT, _INT, _INT, _VP, _LONG, _VP, _LONG]
_SIGNATURES = {
    "gemm_act": (_INT, _SIZES + [_INT, _INT, _VP, _VP, _LONG, _INT, _VP, _LONG, _VP, _LONG, _INT, _VP]),
    "gemm_act_grad": (_INT, _SIZES + [_INT, _INT, _VP, _LONG, _VP, _LONG, _INT, _VP, _VP]),
    "gemm_set_fused_kernel": (_INT, [_INT]),
    "gemm_ce": (_INT, _SIZES + [_FLT, _VP, _VP, _VP, _VP]),
    "gemm_ce_grad": (_INT, _SIZES + [_FLT, _VP, _VP, _VP, _VP, _LONG, _INT, _VP, _LONG, _INT, _FLT, _VP]),
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


def _call(name: str, index: int, stream: Optional[torch.cuda.Stream], *args) -> None:
    """Run entry point ``name`` with ``args`` and the stream on device ``index``;
    switches devices only when another one is current."""
    fn = getattr(_lib or load(), name)
    if index == torch.cuda.current_device():
        status = fn(*args, _stream_handle(stream, index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _stream_handle(stream, index))
    if status != TGEMM_OK:
        raise TgemmError(status, name)


def _activation(act: str) -> int:
    if act not in _ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r}; have {sorted(_ACTIVATIONS)}")
    return _ACTIVATIONS[act]


def _bf16(x, name: str) -> Tuple[int, int, int]:
    """(rows, columns, leading dimension) of a bfloat16 operand. The checks in
    one place and few steps (they are most of a small call's host time); what
    fails them goes to _check_matrix for its error."""
    if isinstance(x, torch.Tensor) and x.dtype is torch.bfloat16 and x.is_cuda:
        shape = x.shape
        if len(shape) == 2:
            rows, cols = shape
            ld, step = x.stride()
            if (step == 1 or cols <= 1) and (ld >= cols or rows <= 1):
                return rows, cols, max(ld, cols, 1)
    ld = _check_matrix(x, name, torch.bfloat16)
    return x.shape[0], x.shape[1], ld


def _operands(A, B, trans_a: bool, trans_b: bool, halves: int):
    """(M, N, K, lda, ldb, flags, device index) of op(A) op(B), whose columns come in ``halves`` halves."""
    rows, cols, lda = _bf16(A, "A")
    M, K = (cols, rows) if trans_a else (rows, cols)
    rows, cols, ldb = _bf16(B, "B")
    K2, wide = (cols, rows) if trans_b else (rows, cols)
    index = A.get_device()
    if index != B.get_device():
        raise ValueError(f"A is on {A.device}, B on {B.device}")
    if K != K2:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} / {tuple(B.shape)}")
    if wide % halves != 0:
        raise ValueError(f"a gated product needs an even number of columns, got {wide}")
    return M, wide // halves, K, lda, ldb, (TGEMM_TRANS_A if trans_a else 0) | (TGEMM_TRANS_B if trans_b else 0), index


def _like(x, name: str, rows: int, cols: int, index: int) -> Tuple[int, int]:
    """(leading dimension, TGEMM_TYPE_*) of a matrix of this shape on this device."""
    if isinstance(x, torch.Tensor) and x.dtype in _TYPES and x.is_cuda and x.shape == (rows, cols) and x.get_device() == index:
        ld, step = x.stride()                 # few steps, as in _bf16
        if (step == 1 or cols <= 1) and (ld >= cols or rows <= 1):
            return max(ld, cols, 1), _TYPES[x.dtype]
    ld, kind = _check_values(x, name)
    if tuple(x.shape) != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected {(rows, cols)}")
    if x.get_device() != index:
        raise ValueError(f"{name} is on {x.device}, the operands on cuda:{index}")
    return ld, kind


def _vector(x, name: str, n: int, dtype: torch.dtype, index: int) -> int:
    """The pointer of a contiguous vector of n elements."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if x.shape != (n,):
        raise ValueError(f"{name} must have {n} elements, got shape {tuple(x.shape)}")
    if not x.is_cuda or x.get_device() != index or (n > 1 and x.stride(0) != 1):
        raise ValueError(f"{name} must be contiguous and on the operands' device")
    return x.data_ptr()


def gemm_act(A: torch.Tensor, B: torch.Tensor, act: str = "none", trans_a: bool = False,
             trans_b: bool = False, gated: bool = False, bias: Optional[torch.Tensor] = None,
             residual: Optional[torch.Tensor] = None, keep_z: bool = False,
             out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None
             ) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """C = act(z) + residual with z = op(A) @ op(B) + bias.

    ``A``/``B`` are the stored bfloat16 matrices, as in :func:`.binding.gemm_ex`:
    A is K x M when ``trans_a`` (else M x K), B is N x K when ``trans_b`` (else
    K x N; a layer's weights kept outputs x inputs take ``trans_b``). ``act`` is
    "none", "relu", "gelu", "gelu_tanh" or "silu". ``gated``: op(B) has 2 N
    columns, C = act(g) * u + residual with [g, u] = z (bfloat16 C). ``bias`` is
    float32, one entry for each column of op(B); ``residual`` M x N, bfloat16 or
    float32, and may be ``out`` itself. With ``keep_z`` (C, Z) comes back, Z the
    bfloat16 z that :func:`gemm_act_grad` takes."""
    code = _activation(act)
    M, N, K, lda, ldb, flags, device = _operands(A, B, trans_a, trans_b, 2 if gated else 1)
    wide = 2 * N if gated else N
    if out is None:
        ldc, kind = max(N, 1), _type(out_dtype, "out_dtype")
    else:
        ldc, kind = _like(out, "out", M, N, device)
    if gated:
        flags |= TGEMM_GATED
        if kind != TGEMM_TYPE_BF16:
            raise TypeError("a gated product's result is bfloat16")
    b = 0 if bias is None else _vector(bias, "bias", wide, torch.float32, device)
    r, ldr, r_kind = 0, 0, 0
    if residual is not None:
        ldr, r_kind = _like(residual, "residual", M, N, device)
        r = residual.data_ptr()
    if out is None:
        out = _empty(stream, M, N, dtype=out_dtype, device=device)
    Z = _empty(stream, M, wide, dtype=torch.bfloat16, device=device) if keep_z else None
    _call("gemm_act", device, stream, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, flags, code, b, r, ldr, r_kind,
          Z.data_ptr() if keep_z else 0, max(wide, 1), out.data_ptr(), ldc, kind)
    return (out, Z) if keep_z else out


def gemm_act_grad(A: torch.Tensor, B: torch.Tensor, Z: torch.Tensor, act: str = "none",
                  trans_a: bool = False, trans_b: bool = False, gated: bool = False,
                  bias_grad: bool = True, out_dtype: torch.dtype = torch.bfloat16,
                  out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                  ) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """dZ = d * act'(Z) with d = op(A) @ op(B), and db, its column sums (float32).

    Takes the gradient A of the next layer's output through that layer's weights
    B (kept outputs x inputs: no flags) and through the activation that made its
    input; Z is what :func:`gemm_act` kept. ``gated``: Z = [g, u] and dZ = [d * u *
    act'(g), d * act(g)] have 2 N columns. dZ goes to ``out`` (which may be Z) or
    a new ``out_dtype`` matrix; without ``bias_grad`` only dZ comes back."""
    code = _activation(act)
    M, N, K, lda, ldb, flags, device = _operands(A, B, trans_a, trans_b, 1)
    wide = 2 * N if gated else N
    ldz, z_kind = _like(Z, "Z", M, wide, device)
    if z_kind != TGEMM_TYPE_BF16:
        raise TypeError("Z must be bfloat16")
    if out is None:
        ldc, kind = max(wide, 1), _type(out_dtype, "out_dtype")
    else:
        ldc, kind = _like(out, "out", M, wide, device)
    if gated:
        flags |= TGEMM_GATED
        if kind != z_kind:
            raise TypeError("a gated product's gradient is bfloat16")
    if out is None:
        out = _empty(stream, M, wide, dtype=out_dtype, device=device)
    db = _empty(stream, wide, dtype=torch.float32, device=device) if bias_grad else None
    _call("gemm_act_grad", device, stream, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, flags, code, Z.data_ptr(), ldz,
          out.data_ptr(), ldc, kind, db.data_ptr() if bias_grad else 0)
    return (out, db) if bias_grad else out


def _head(X, W, target):
    """(T, V, D, ldx, ldw, target's pointer, device index) of a head's product."""
    T, D, ldx = _bf16(X, "X")
    V, D2, ldw = _bf16(W, "W")
    index = X.get_device()
    if index != W.get_device():
        raise ValueError(f"X is on {X.device}, W on {W.device}")
    if D != D2:
        raise ValueError(f"inner dimensions differ: {tuple(X.shape)} / {tuple(W.shape)}")
    return T, V, D, ldx, ldw, _vector(target, "target", T, torch.int64, index), index


def gemm_ce(X: torch.Tensor, W: torch.Tensor, target: torch.Tensor, alpha: float = 1.0,
            stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(loss, lse), float32, of T tokens over a vocabulary of V entries: with the
    logits z = alpha * X @ W.T, lse = log sum exp z of each row and loss = lse -
    z[target]. X (T x D) and W (V x D) are bfloat16, target int64; a row whose
    target is not in 0 .. V - 1 is left out, with a loss of 0. The logits are
    not kept."""
    T, V, D, ldx, ldw, t, device = _head(X, W, target)
    loss = _empty(stream, T, dtype=torch.float32, device=device)
    lse = _empty(stream, T, dtype=torch.float32, device=device)
    _call("gemm_ce", device, stream, T, V, D, X.data_ptr(), ldx, W.data_ptr(), ldw, alpha, t, loss.data_ptr(),
          lse.data_ptr())
    return loss, lse


def gemm_ce_grad(X: torch.Tensor, W: torch.Tensor, target: torch.Tensor, lse: torch.Tensor,
                 dloss: torch.Tensor, alpha: float = 1.0, x_grad: bool = True, w_grad: bool = True,
                 dx_dtype: torch.dtype = torch.bfloat16, dw_dtype: torch.dtype = torch.bfloat16,
                 dw_out: Optional[torch.Tensor] = None, beta: float = 0.0,
                 stream: Optional[torch.cuda.Stream] = None
                 ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dX, dW), the gradients of sum(dloss * loss) of :func:`gemm_ce` with its lse
    (``dloss`` float32, one entry a token). The logits' gradient is rounded to bfloat16
    between the products, for float32 results too. ``x_grad``/``w_grad`` say which are
    wanted (the other is None). dW goes to ``dw_out``, plus ``beta`` times what
    is there (a sum over micro-batches), or to a new ``dw_dtype`` matrix."""
    T, V, D, ldx, ldw, t, device = _head(X, W, target)
    lse_ptr = _vector(lse, "lse", T, torch.float32, device)
    dloss_ptr = _vector(dloss, "dloss", T, torch.float32, device)
    dx, dw, x_kind, w_kind, lddx, lddw = None, None, 0, 0, D, D
    if dw_out is None and beta != 0.0:
        raise ValueError("beta != 0 needs dw_out, the dW it scales")
    if dw_out is not None and not w_grad:
        raise ValueError("dw_out without w_grad")
    if x_grad:
        x_kind = _type(dx_dtype, "dx_dtype")
    if w_grad and dw_out is None:
        w_kind = _type(dw_dtype, "dw_dtype")
    elif w_grad:
        lddw, w_kind = _like(dw_out, "dw_out", V, D, device)
        dw = dw_out
    if x_grad:
        dx = _empty(stream, T, D, dtype=dx_dtype, device=device)
    if w_grad and dw is None:
        dw = _empty(stream, V, D, dtype=dw_dtype, device=device)
    _call("gemm_ce_grad", device, stream, T, V, D, X.data_ptr(), ldx, W.data_ptr(), ldw, alpha, t, lse_ptr, dloss_ptr,
          dx.data_ptr() if x_grad else 0, lddx, x_kind, dw.data_ptr() if w_grad else 0, lddw, w_kind, beta)
    return dx, dw


def set_fused_kernel(mode: int) -> int:
    """-1: by a model of the kernels' times; 0: 256 x 256 tiles on SM pairs; 1: few
    tiles, on one SM each."""
    return int(load().gemm_set_fused_kernel(int(mode)))
