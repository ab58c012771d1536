"""ctypes binding of libhpo's model operators (include/hpo_model.h).

As in `hpo` and `hpo_stack`: every entry point keeps its C name, torch tensors
stand where the C call takes device memory, `stream=None` means torch's current
stream, and nothing here computes on the data.  A stack is a tensor
[batch, rows, cols] or [rows, cols] whose last dimension is contiguous; an
8-bit one is float8_e4m3fn with its block scales (uint8 or float8_e8m0fnu, of
hpo_stack.mx_scales_shape) beside it.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import hpo
from .hpo import HPO_OK, _check
from .hpo_stack import (_SCALE_DTYPES, _buffer, _device, _shape3, _stack, _stream, _workspace, c_stack,
                        mx_scales_shape)

_P, _I32, _I64, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_S = ctypes.POINTER(c_stack)
_OUT = ctypes.POINTER(_I64)

# name -> (restype, argtypes), exactly as declared in include/hpo_model.h
SIGNATURES = {
    "hpo_embedding": (_I32, [_P, _I32, _I64, _I64, _S, _P, _F32, _S, _P]),
    "hpo_embedding_grad": (_I32, [_P, _I32, _I64, _I64, _S, _F32, _S, _P, _I64, _P]),
    "hpo_embedding_grad_workspace": (_I32, [_I64, _I64, _OUT]),
    "hpo_mx8_save": (_I32, [_S, _S, _P, _P]),
    "hpo_mx8_linear": (_I32, [_S, _P, _S, _P, _S, _P, _I64, _P]),
    "hpo_mx8_dgrad": (_I32, [_S, _S, _P, _S, _P, _I64, _P]),
    "hpo_mx8_wgrad": (_I32, [_S, _S, _P, _F32, _I32, _S, _P, _I64, _P]),
    "hpo_mx8_linear_workspace": (_I32, [_I64, _I64, _I64, _I64, _OUT]),
    "hpo_mx8_dgrad_workspace": (_I32, [_I64, _I64, _I64, _I64, _OUT]),
    "hpo_mx8_wgrad_workspace": (_I32, [_I64, _I64, _I64, _I64, _OUT]),
}

_lib = None


def load():
    global _lib
    if _lib is None:
        lib = hpo.load()
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _scales(scales: Optional[torch.Tensor], t: torch.Tensor, what: str, dev: int):
    """Address of the block scales of t; None where none are given."""
    if scales is None:
        return None
    if scales.dtype not in _SCALE_DTYPES:
        raise TypeError(f"{what} must be uint8 or float8_e8m0fnu, got {scales.dtype}")
    return _buffer(scales, what, dev, None, math.prod(mx_scales_shape(t)))


def _ids(ids: torch.Tensor, dev: int):
    """(address, bytes of one, how many) of the token ids."""
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    return _buffer(ids, "ids", dev, None, 0), ids.element_size(), ids.numel()


def _rows(t: torch.Tensor, n: int, what: str) -> torch.Tensor:
    """t with one row per token: [..., cols], as [n, cols] without a copy."""
    if t.dim() == 2:
        return t
    if t.dim() < 1 or math.prod(t.shape[:-1]) != n:
        raise ValueError(f"{what} must hold one row for each of the {n} ids, got {tuple(t.shape)}")
    try:
        return t.view(n, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"{what}: the rows of {tuple(t.shape)} do not lie at one stride") from None


# --------------------------------------------------------------------------
# entry points (same names as the C ABI)
# --------------------------------------------------------------------------
def hpo_embedding(ids: torch.Tensor, weight: torch.Tensor, out: torch.Tensor, scales: Optional[torch.Tensor] = None,
                  scale: float = 1.0, first: int = 0, stream=None) -> None:
    """out[..., :] = scale * weight[ids - first], zeros for ids outside the table.  ids: int32 or
    int64 of any shape, contiguous; weight [rows, cols] bf16, fp16, fp32, or float8_e4m3fn with
    scales; out [*ids.shape, cols] (or [ids.numel(), cols]) bf16, fp16 or fp32."""
    dev = _device()
    at, nbytes, n = _ids(ids, dev)
    st = load().hpo_embedding(at, nbytes, n, first, ctypes.byref(_stack(weight, "weight", dev)),
                              _scales(scales, weight, "scales", dev), scale,
                              ctypes.byref(_stack(_rows(out, n, "out"), "out", dev)), _stream(stream, dev))
    if st != HPO_OK:
        _check(st, "hpo_embedding")


def hpo_embedding_grad_workspace(ids: torch.Tensor, grad: torch.Tensor) -> int:
    """Bytes of workspace for as many ids and rows as wide as grad's."""
    out = _I64()
    _check(load().hpo_embedding_grad_workspace(ids.numel(), grad.shape[-1], ctypes.byref(out)),
           "hpo_embedding_grad_workspace")
    return out.value


def hpo_embedding_grad(ids: torch.Tensor, dy: torch.Tensor, grad: torch.Tensor, workspace: Optional[torch.Tensor],
                       scale: float = 1.0, first: int = 0, stream=None) -> None:
    """grad[ids - first] += scale * dy (fp32 or bf16 main grad, in place), every token's row once;
    ids outside the table count for nothing.  dy: bf16, fp16 or fp32, [*ids.shape, cols]."""
    dev = _device()
    at, nbytes, n = _ids(ids, dev)
    ws, size = _workspace(workspace, dev)
    st = load().hpo_embedding_grad(at, nbytes, n, first, ctypes.byref(_stack(_rows(dy, n, "dy"), "dy", dev)), scale,
                                   ctypes.byref(_stack(grad, "grad", dev)), ws, size, _stream(stream, dev))
    if st != HPO_OK:
        _check(st, "hpo_embedding_grad")


def hpo_mx8_save(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """q (float8_e4m3fn) and scales = x (bf16, fp16 or fp32) in 8 bits with block scales."""
    dev = _device()
    st = load().hpo_mx8_save(ctypes.byref(_stack(x, "x", dev)), ctypes.byref(_stack(q, "q", dev)),
                             _scales(scales, q, "scales", dev), _stream(stream, dev))
    if st != HPO_OK:
        _check(st, "hpo_mx8_save")


def _product_workspace(name: str, batch: int, tokens: int, cols: int, rows: int) -> int:
    out = _I64()
    _check(getattr(load(), name)(batch, tokens, cols, rows, ctypes.byref(out)), name)
    return out.value


def hpo_mx8_linear_workspace(x: torch.Tensor, w: torch.Tensor) -> int:
    (b, t, c), r = _shape3(x), w.shape[-2]
    return _product_workspace("hpo_mx8_linear_workspace", b, t, c, r)


def hpo_mx8_dgrad_workspace(dy: torch.Tensor, w: torch.Tensor) -> int:
    (b, t, r), c = _shape3(dy), w.shape[-1]
    return _product_workspace("hpo_mx8_dgrad_workspace", b, t, c, r)


def hpo_mx8_wgrad_workspace(dy: torch.Tensor, x: torch.Tensor) -> int:
    (b, t, r), c = _shape3(dy), x.shape[-1]
    return _product_workspace("hpo_mx8_wgrad_workspace", b, t, c, r)


def hpo_mx8_linear(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, y: torch.Tensor,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """y [tokens, rows] (bf16 or fp16) = x [tokens, cols] times the transpose of w [rows, cols], both
    in 8 bits; each may have a leading batch dimension."""
    dev = _device()
    ws, size = _workspace(workspace, dev)
    st = load().hpo_mx8_linear(ctypes.byref(_stack(x, "x", dev)), _scales(x_scales, x, "x_scales", dev),
                               ctypes.byref(_stack(w, "w", dev)), _scales(w_scales, w, "w_scales", dev),
                               ctypes.byref(_stack(y, "y", dev)), ws, size, _stream(stream, dev))
    if st != HPO_OK:
        _check(st, "hpo_mx8_linear")


def hpo_mx8_dgrad(dy: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, dx: torch.Tensor,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """dx [tokens, cols] (bf16, fp16 or fp32) = dy [tokens, rows] (bf16 or fp16) times w [rows, cols]."""
    dev = _device()
    ws, size = _workspace(workspace, dev)
    st = load().hpo_mx8_dgrad(ctypes.byref(_stack(dy, "dy", dev)), ctypes.byref(_stack(w, "w", dev)),
                              _scales(w_scales, w, "w_scales", dev), ctypes.byref(_stack(dx, "dx", dev)), ws, size,
                              _stream(stream, dev))
    if st != HPO_OK:
        _check(st, "hpo_mx8_dgrad")


def hpo_mx8_wgrad(dy: torch.Tensor, x: torch.Tensor, x_scales: torch.Tensor, grad: torch.Tensor,
                  workspace: Optional[torch.Tensor] = None, scale: float = 1.0, accumulate: bool = True,
                  stream=None) -> None:
    """grad [rows, cols] (fp32 or bf16 main grad) += scale * (transpose of dy [tokens, rows]) times
    x [tokens, cols], or = with accumulate=False."""
    dev = _device()
    ws, size = _workspace(workspace, dev)
    st = load().hpo_mx8_wgrad(ctypes.byref(_stack(dy, "dy", dev)), ctypes.byref(_stack(x, "x", dev)),
                              _scales(x_scales, x, "x_scales", dev), scale, 1 if accumulate else 0,
                              ctypes.byref(_stack(grad, "grad", dev)), ws, size, _stream(stream, dev))
    if st != HPO_OK:
        _check(st, "hpo_mx8_wgrad")
