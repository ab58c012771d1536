"""ctypes binding of libhpo's stack operators (include/hpo_stack.h).

As in `hpo`: every entry point keeps its C name, torch tensors stand where the
C call takes device memory, `stream=None` means torch's current stream, and
nothing here computes on the data.  A stack is a tensor [batch, rows, cols] or
[rows, cols] (one matrix) whose last dimension is contiguous; its other strides
are free within the rules of the C call.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional, Sequence

import torch

from . import hpo
from .hpo import HPO_OK, HPO_PARAM_BF16, HPO_PARAM_FP16, HPO_PARAM_FP32, _check

HPO_WEIGHT_MX8 = 16
HPO_QK_MAX_DIM = 256
HPO_CLIP_MAX_WEIGHTS = 8
MX_BLOCK = 32

_P, _I32, _I64, _F64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double


class c_stack(ctypes.Structure):
    _fields_ = [("data", _P), ("batch", _I64), ("rows", _I64), ("cols", _I64), ("batch_stride", _I64),
                ("row_stride", _I64), ("dtype", _I32), ("reserved", _I32)]


class hpo_rms_cfg(ctypes.Structure):
    _fields_ = [("lr", _F64), ("weight_decay", _F64), ("beta2", _F64), ("eps", _F64), ("target_rms", _F64)]


class c_qk(ctypes.Structure):
    _fields_ = [("q", _P), ("k", _P), ("dtype", _I32), ("batch", _I32), ("heads", _I32), ("kv_heads", _I32),
                ("head_dim", _I32), ("causal", _I32), ("window", _I64), ("seq_q", _I64), ("seq_k", _I64),
                ("max_seqlen_q", _I64), ("max_seqlen_k", _I64),
                ("q_stride_batch", _I64), ("q_stride_token", _I64), ("q_stride_head", _I64),
                ("k_stride_batch", _I64), ("k_stride_token", _I64), ("k_stride_head", _I64),
                ("cu_seqlens_q", _P), ("cu_seqlens_k", _P), ("seqlens_q", _P), ("seqlens_k", _P),
                ("scale", ctypes.c_float), ("reserved", _I32)]


class c_clip_weight(ctypes.Structure):
    _fields_ = [("master", ctypes.POINTER(c_stack)), ("param", ctypes.POINTER(c_stack)), ("d_scales", _P),
                ("power", _F64), ("per_group", _I32), ("reserved", _I32)]


_S = ctypes.POINTER(c_stack)

# name -> (restype, argtypes), exactly as declared in include/hpo_stack.h
SIGNATURES = {
    "hpo_orthogonalize": (_I32, [_S, _S, _S, ctypes.POINTER(hpo.hpo_muon_cfg), ctypes.c_float, _F64, _P, _P, _P, _I64,
                                 _P]),
    "hpo_orthogonalize_workspace": (_I32, [_I64, _I64, _I64, ctypes.POINTER(_I64)]),
    "hpo_rms_update": (_I32, [_S, _S, _P, _S, _P, ctypes.POINTER(hpo_rms_cfg), _P, _P, _I64, _P]),
    "hpo_rms_update_workspace": (_I32, [_I64, _I64, ctypes.POINTER(_I64)]),
    "hpo_qk_max_logits": (_I32, [ctypes.POINTER(c_qk), _I32, _P, _P]),
    "hpo_qk_clip": (_I32, [_P, _I32, _I32, _F64, ctypes.POINTER(c_clip_weight), _I32, _P, _P]),
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


_CODES = {torch.float32: HPO_PARAM_FP32, torch.bfloat16: HPO_PARAM_BF16, torch.float16: HPO_PARAM_FP16,
          torch.float8_e4m3fn: HPO_WEIGHT_MX8}


# These calls are a few microseconds of work on small weights, so what is done
# per call here is kept short: one look at the current device, plain integers
# for pointers and the stream.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _device() -> int:
    """The current device, or -1 without one (every tensor is then refused)."""
    return torch.cuda.current_device() if torch.cuda.is_initialized() or torch.cuda.is_available() else -1


def _stream(stream, dev: int):
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return hpo._stream(stream)


def _refuse_device(t: torch.Tensor, what: str, dev: int):
    if t.get_device() < 0:
        raise ValueError(f"{what} must be a device tensor")
    raise ValueError(f"{what} is on {t.device} but the current device is cuda:{dev}")


def _stack(t: torch.Tensor, what: str, dev: int) -> c_stack:
    at = t.get_device()
    if at != dev or at < 0:
        _refuse_device(t, what, dev)
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: {t.dtype} is not supported")
    shape, strides = t.shape, t.stride()
    if len(shape) == 3:
        b, r, c = shape
        bs, rs, cs = strides
    elif len(shape) == 2:
        b, bs = 1, 0
        r, c = shape
        rs, cs = strides
    else:
        raise ValueError(f"{what} must have 2 or 3 dimensions, got {len(shape)}")
    if cs != 1 and c > 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return c_stack(t.data_ptr(), b, r, c, bs, rs, code, 0)


def _opt(t: Optional[torch.Tensor], what: str, dev: int):
    return None if t is None else ctypes.byref(_stack(t, what, dev))


def _buffer(t, what: str, dev: int, dtype, min_bytes: int):
    """Address of a contiguous device buffer; None is NULL, an int a raw address."""
    if t is None or isinstance(t, int):
        return t
    at = t.get_device()
    if at != dev or at < 0:
        _refuse_device(t, what, dev)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() * t.element_size() < min_bytes:
        raise ValueError(f"{what} spans {t.numel() * t.element_size()} bytes, the call needs {min_bytes}")
    return t.data_ptr()


def _workspace(t: Optional[torch.Tensor], dev: int):
    return (None, 0) if t is None else (_buffer(t, "workspace", dev, None, 0), t.numel() * t.element_size())


def _shape3(t: torch.Tensor):
    return tuple(t.shape) if t.dim() == 3 else (1, *t.shape)


def mx_scales_shape(t: torch.Tensor):
    """Shape of the block scales of a stack held in 8 bits: one per 32 elements of a row."""
    b, r, c = _shape3(t)
    s = (b, r, -(-c // MX_BLOCK))
    return s if t.dim() == 3 else s[1:]


_SCALE_DTYPES = (torch.uint8, getattr(torch, "float8_e8m0fnu", torch.uint8))


def _scales_ptr(scales: Optional[torch.Tensor], param: Optional[torch.Tensor], what: str, dev: int):
    if scales is None:
        return None
    if scales.dtype not in _SCALE_DTYPES:
        raise TypeError(f"{what} must be uint8 or float8_e8m0fnu, got {scales.dtype}")
    if param is None:
        raise ValueError(f"{what} without a param")
    return _buffer(scales, what, dev, None, math.prod(mx_scales_shape(param)))


# --------------------------------------------------------------------------
# entry points (same names as the C ABI)
# --------------------------------------------------------------------------
def hpo_orthogonalize_workspace(G: torch.Tensor, cfg=None, momentum: Optional[torch.Tensor] = None) -> int:
    """Bytes of workspace for a stack of G's shape (cfg and momentum do not change it)."""
    out = _I64()
    _check(load().hpo_orthogonalize_workspace(*_shape3(G), ctypes.byref(out)), "hpo_orthogonalize_workspace")
    return out.value


def hpo_orthogonalize(G: torch.Tensor, out: torch.Tensor, cfg: hpo.hpo_muon_cfg, workspace: Optional[torch.Tensor],
                      momentum: Optional[torch.Tensor] = None, inv_scale: float = 1.0, max_norm: float = 0.0,
                      d_norm=None, d_found_inf=None, stream=None) -> None:
    """out (bf16) = the orthogonalised Nesterov gradient of every matrix of G
    (fp32 or bf16); momentum (fp32, in place) may be left out.  The workspace is a
    uint8 device tensor of hpo_orthogonalize_workspace bytes."""
    dev = _device()
    ws, nbytes = _workspace(workspace, dev)
    st = load().hpo_orthogonalize(ctypes.byref(_stack(G, "G", dev)), _opt(momentum, "momentum", dev),
                                  ctypes.byref(_stack(out, "out", dev)), ctypes.byref(cfg), inv_scale, max_norm,
                                  _buffer(d_norm, "d_norm", dev, torch.float32, 4),
                                  _buffer(d_found_inf, "d_found_inf", dev, torch.int32, 4), ws, nbytes,
                                  _stream(stream, dev))
    if st != HPO_OK:
        _check(st, "hpo_orthogonalize")


def make_rms_cfg(lr: float, weight_decay: float = 0.0, beta2: float = 0.95, eps: float = 1e-8,
                 target_rms: float = 0.2) -> hpo_rms_cfg:
    """target_rms 0.2 is the update size of Moonlight's 0.2 sqrt(max(A, B)) scale."""
    return hpo_rms_cfg(lr, weight_decay, beta2, eps, target_rms)


def hpo_rms_update_workspace(master: torch.Tensor) -> int:
    out = _I64()
    b, r, _ = _shape3(master)
    _check(load().hpo_rms_update_workspace(b, r, ctypes.byref(out)), "hpo_rms_update_workspace")
    return out.value


def hpo_rms_update(O: torch.Tensor, master: torch.Tensor, v: Optional[torch.Tensor], cfg: hpo_rms_cfg,
                   workspace: Optional[torch.Tensor], param: Optional[torch.Tensor] = None,
                   scales: Optional[torch.Tensor] = None, d_found_inf=None, stream=None) -> None:
    """Row-normalised update of master (fp32, in place) by O (bf16 or fp32), with v
    (fp32 [batch, rows]) its running row mean squares, and the model weight:
    bf16, or float8_e4m3fn with scales (uint8 / float8_e8m0fnu, mx_scales_shape)."""
    dev = _device()
    ws, nbytes = _workspace(workspace, dev)
    w = _stack(master, "master", dev)
    st = load().hpo_rms_update(ctypes.byref(_stack(O, "O", dev)), ctypes.byref(w),
                               _buffer(v, "v", dev, torch.float32, 4 * w.batch * w.rows), _opt(param, "param", dev),
                               _scales_ptr(scales, param, "scales", dev), ctypes.byref(cfg),
                               _buffer(d_found_inf, "d_found_inf", dev, torch.int32, 4), ws, nbytes,
                               _stream(stream, dev))
    if st != HPO_OK:
        _check(st, "hpo_rms_update")


def hpo_qk_max_logits(q: torch.Tensor, k: torch.Tensor, d_max: torch.Tensor, scale: float, causal: bool = True,
                      window: int = -1, cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q: Optional[int] = None,
                      max_seqlen_k: Optional[int] = None, seqlens_q=None, seqlens_k=None, accumulate: bool = False,
                      stream=None) -> None:
    """d_max[h] (fp32) = the largest scale * (q . k) that head h sees.  q, k: bf16 or
    fp16, [batch, tokens, heads, dim] (seqlens_* int32 [batch] cut the batch rows), or
    packed [tokens, heads, dim] with cu_seqlens_* int32 [batch + 1]."""
    dev = _device()
    packed = cu_seqlens_q is not None or cu_seqlens_k is not None
    dims = 3 if packed else 4
    code = _CODES.get(q.dtype)
    for what, t in (("q", q), ("k", k)):
        if t.get_device() != dev or dev < 0:
            _refuse_device(t, what, dev)
        if t.dim() != dims:
            raise ValueError(f"{what} must have {dims} dimensions, got {t.dim()}")
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"{what}: the last dimension must be contiguous")
    if code is None:
        raise TypeError(f"q: {q.dtype} is not supported")
    qs, ks = q.shape, k.shape
    if q.dtype != k.dtype or qs[-1] != ks[-1] or (not packed and qs[0] != ks[0]):
        raise ValueError(f"q {tuple(qs)} {q.dtype} and k {tuple(ks)} {k.dtype} do not go together")
    if packed:
        if cu_seqlens_q is None or cu_seqlens_k is None or max_seqlen_q is None or max_seqlen_k is None:
            raise ValueError("packed sequences need cu_seqlens_q, cu_seqlens_k, max_seqlen_q and max_seqlen_k")
        batch = cu_seqlens_q.numel() - 1
        if batch < 0 or cu_seqlens_k.numel() != batch + 1:
            raise ValueError("cu_seqlens_q and cu_seqlens_k must hold batch + 1 offsets each")
        qst, kst = (0, *q.stride()), (0, *k.stride())
    else:
        batch, qst, kst = qs[0], q.stride(), k.stride()
    lens = [None if t is None else _buffer(t, what, dev, torch.int32, n)
            for t, what, n in ((cu_seqlens_q, "cu_seqlens_q", 4 * batch + 4), (cu_seqlens_k, "cu_seqlens_k", 4 * batch + 4),
                               (seqlens_q, "seqlens_q", 4 * batch), (seqlens_k, "seqlens_k", 4 * batch))]
    a = c_qk(q.data_ptr(), k.data_ptr(), code, batch, qs[-2], ks[-2], qs[-1], 1 if causal else 0, window, qs[-3],
             ks[-3], max_seqlen_q or 0, max_seqlen_k or 0, qst[0], qst[1], qst[2], kst[0], kst[1], kst[2], *lens,
             scale, 0)
    st = load().hpo_qk_max_logits(ctypes.byref(a), 1 if accumulate else 0,
                                  _buffer(d_max, "d_max", dev, torch.float32, 4 * qs[-2]), _stream(stream, dev))
    if st != HPO_OK:
        _check(st, "hpo_qk_max_logits")


class ClipWeight(NamedTuple):
    """A weight that QK-clip rescales: `master` (fp32) is [heads * dim, cols] or
    [heads, dim, cols], one matrix per head; `param` (bf16, or float8_e4m3fn with
    `scales`) has the same shape; gamma enters to the `power`."""
    master: torch.Tensor
    heads: int
    power: float
    param: Optional[torch.Tensor] = None
    scales: Optional[torch.Tensor] = None
    per_group: bool = True


def _head_stack(t: torch.Tensor, heads: int, what: str, dev: int) -> c_stack:
    """t as a stack of one matrix per head: [heads * dim, cols] or [heads, dim, cols]."""
    s = _stack(t, what, dev)
    if t.dim() == 2:
        if heads < 1 or s.rows % heads:
            raise ValueError(f"{what}: {s.rows} rows are not {heads} heads")
        s.batch, s.rows = heads, s.rows // heads
        s.batch_stride = s.rows * s.row_stride
    elif s.batch != heads:
        raise ValueError(f"{what} must be [{heads} * dim, cols] or [{heads}, dim, cols], got {tuple(t.shape)}")
    return s


def hpo_qk_clip(d_max: torch.Tensor, kv_heads: int, tau: float, weights: Sequence[ClipWeight], d_found_inf=None,
                stream=None) -> None:
    """Rescales the rows of the heads whose d_max is over tau (in place)."""
    dev = _device()
    n = len(weights)
    arr = (c_clip_weight * max(n, 1))()
    keep = []
    for k, w in enumerate(weights):
        what = f"weights[{k}]."
        ms = _head_stack(w.master, w.heads, what + "master", dev)
        keep.append(ms)
        c = arr[k]
        c.master = ctypes.pointer(ms)
        if w.param is not None:
            ps = _head_stack(w.param, w.heads, what + "param", dev)
            keep.append(ps)
            c.param = ctypes.pointer(ps)
        if w.scales is not None:
            c.d_scales = _scales_ptr(w.scales, w.param, what + "scales", dev)
        c.power = w.power
        c.per_group = 1 if w.per_group else 0
    heads = d_max.numel()
    st = load().hpo_qk_clip(_buffer(d_max, "d_max", dev, torch.float32, 4 * heads), heads, kv_heads, tau, arr, n,
                            _buffer(d_found_inf, "d_found_inf", dev, torch.int32, 4), _stream(stream, dev))
    if st != HPO_OK:
        _check(st, "hpo_qk_clip")
