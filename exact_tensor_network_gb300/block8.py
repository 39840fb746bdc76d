"""Matrices in 8 bits with a scale for each block of 128, and their products
(``include/tn_block8.h``).

The functions with the C names only marshal arguments; the others work on torch
tensors.  ``Blocks8`` is a quantised matrix: codes (float8_e4m3fn [rows, cols], rows
starting at multiples of 16 bytes) and scales (float32, [rows, blocks] or, for
blocks of 128 x 128 entries, [blocks of rows, blocks], of any strides; ``quantize8``
lays those of rows out with the rows next to each other, which products read fastest).

    w = quantize8(weight, square=True)              # a head's weights, kept in 8 bits
    y = linear8(x, w)                               # rows of logits
    wt = quantize8(weight, square=True, layout="columns")
    dx, dw = linear8_grad(x, dy, wt)                # and their gradients

All tensors of a call and its stream are on the current device.  Calls are
asynchronous on ``stream`` (default: torch's current stream); on another stream
the caller orders it after the inputs' producers, the inputs and outputs are recorded
on it, and what the call makes belongs to it.  Nothing is recorded for automatic
differentiation: ``linear8_grad`` is the backward pass.  Every call runs in the
library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple

from .outcomes import TN_TYPE_BF16, TN_TYPE_F16, TN_TYPE_F32

_P = ctypes.c_void_p
_I32, _I64 = ctypes.c_int32, ctypes.c_int64

TN_BLOCK8 = 128


class tn_matrix(ctypes.Structure):
    _fields_ = [("data", _P), ("type", _I32), ("rows", _I64), ("cols", _I64), ("row_stride", _I64),
                ("col_stride", _I64)]


class tn_block8(ctypes.Structure):
    _fields_ = [("codes", _P), ("scales", _P), ("rows", _I64), ("cols", _I64), ("row_stride", _I64),
                ("scale_stride", _I64), ("scale_block", _I64), ("block_rows", _I32), ("powers", _I32)]


_MP, _BP = ctypes.POINTER(tn_matrix), ctypes.POINTER(tn_block8)

# exported symbol -> (restype, argtypes)
SIGNATURES = {
    "tn_block8_quantize": (ctypes.c_int, [_MP, _BP, _BP, _P]),
    "tn_block8_product": (ctypes.c_int, [_BP, _BP, _P, _I32, _I64, _P]),
    "tn_block8_check": (ctypes.c_int, []),
    "tn_block8_last_error": (ctypes.c_char_p, []),
}


_L = None           # the library, looked up once: small calls cost what their host side costs


def _lib():
    global _L
    if _L is None:
        from . import lib
        _L = lib()
    return _L


def _check(st: int) -> None:
    if st != 0:
        from . import TNError, tn_status_string
        raise TNError(st, tn_block8_last_error() or tn_status_string(st))


# ---- functions with the C names -------------------------------------------

def tn_block8_quantize(x: tn_matrix, rows, columns, stream: int = 0) -> None:
    """``rows`` and ``columns`` are ``tn_block8`` or None."""
    _check(_lib().tn_block8_quantize(x, rows, columns, stream))


def tn_block8_product(a: tn_block8, b: tn_block8, out: int, type_: int, out_stride: int, stream: int = 0) -> None:
    _check(_lib().tn_block8_product(a, b, out, type_, out_stride, stream))


def tn_block8_check() -> None:
    _check(_lib().tn_block8_check())


def tn_block8_last_error() -> str:
    return _lib().tn_block8_last_error().decode()


# ---- over torch tensors ----------------------------------------------------

class Blocks8(NamedTuple):
    """A quantised matrix: ``codes`` and ``scales``.  ``powers``: the scales are
    powers of two (or NaN), as ``quantize8`` makes them and products are faster with;
    False for any float32 scales."""
    codes: object
    scales: object
    powers: bool = True

    def values(self):
        """What the codes stand for, in float32 (by torch, for inspection)."""
        c = self.codes.float()
        s = self.scales
        if s.shape[0] != c.shape[0]:
            s = s.repeat_interleave(TN_BLOCK8, 0)[:c.shape[0]]
        return c * s.repeat_interleave(TN_BLOCK8, 1)[:, :c.shape[1]]


_TORCH = _TYPES = _F8 = _F32 = None     # torch, torch dtype -> TN_TYPE_*, two of its types


def _types():
    global _TORCH, _TYPES, _F8, _F32
    if _TYPES is None:
        import torch
        _TORCH, _F8, _F32 = torch, torch.float8_e4m3fn, torch.float32
        _TYPES = {torch.float32: TN_TYPE_F32, torch.bfloat16: TN_TYPE_BF16, torch.float16: TN_TYPE_F16}
    return _TYPES


def _matrix(t, name) -> tn_matrix:
    type_ = _types().get(t.dtype)
    shape = t.shape
    if type_ is None or not t.is_cuda or len(shape) != 2:
        raise ValueError(f"{name} must be a 2-dimensional float32, bfloat16 or float16 CUDA tensor")
    if t.is_neg():
        raise ValueError(f"{name} is a lazily negated view: resolve it first")
    if t.device.index != _TORCH._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, which is not the current device")
    return tn_matrix(t.data_ptr(), type_, *shape, *t.stride())


def _blocks(b, name, device) -> tn_block8:
    _types()
    codes, scales, powers = b
    shape, sshape = codes.shape, scales.shape
    if codes.dtype is not _F8 or len(shape) != 2 or codes.device != device:
        raise ValueError(f"codes of {name} must be a 2-dimensional float8_e4m3fn tensor on the other operands' device")
    R, C = shape
    stride, step = codes.stride()
    if C > 1 and step != 1:
        raise ValueError(f"rows of the codes of {name} must be contiguous")
    blocks = -(-C // TN_BLOCK8)
    if scales.dtype is not _F32 or scales.device != device or len(sshape) != 2 or scales.is_neg():
        raise ValueError(f"scales of {name} must be a float32 matrix on the codes' device")
    tall = -(-R // TN_BLOCK8)
    if sshape[1] != blocks or (sshape[0] != R and sshape[0] != tall):
        raise ValueError(f"scales of {name} must be [{R}, {blocks}] or [{tall}, {blocks}], not {tuple(sshape)}")
    # one row, or empty ones, have no stride of their own
    if R <= 1 or C == 0:
        stride = -(-C // 16) * 16
    row, block = scales.stride()
    return tn_block8(codes.data_ptr(), scales.data_ptr(), R, C, stride, row if sshape[0] > 1 else 1,
                     block if blocks > 1 else 1, 1 if sshape[0] == R else TN_BLOCK8, 1 if powers else 0)


_HERE = contextlib.nullcontext()


def _stream(device, stream, tensors):
    """(stream handle, what makes tensors on it)."""
    torch = _TORCH
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index), _HERE
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    elif getattr(stream, "device", device) != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream, torch.cuda.stream(stream)


def _new(R, C, square, device):
    """(a new matrix, its tn_block8)."""
    stride, blocks = -(-C // 16) * 16, -(-C // TN_BLOCK8)
    codes = _TORCH.empty((R, stride), dtype=_F8, device=device)
    if square:
        tall = -(-R // TN_BLOCK8)
        scales = _TORCH.empty((tall, blocks), dtype=_F32, device=device)
        row, block = max(blocks, 1), 1
    else:
        scales = _TORCH.empty_strided((R, blocks), (1, max(R, 1)), dtype=_F32, device=device)
        row, block = 1, max(R, 1)
    b = tn_block8(codes.data_ptr(), scales.data_ptr(), R, C, stride, row, block, TN_BLOCK8 if square else 1, 1)
    return Blocks8(codes if stride == C else codes[:, :C], scales), b


class _Scratch:
    """Codes and scales of a call's own, in one allocation."""

    def __init__(self, R, C, device):
        stride, blocks = -(-C // 16) * 16, -(-C // TN_BLOCK8)
        self.memory = _TORCH.empty(R * (stride + 4 * blocks), dtype=_TORCH.uint8, device=device)
        p = self.memory.data_ptr()
        self.blocks = tn_block8(p, p + R * stride, R, C, stride, 1, max(R, 1), 1, 1)


def quantize8(x, square: bool = False, layout: str = "rows", out=None, stream=None):
    """``x`` ([R, C], any strides) in 8 bits.  ``square``: a scale for 128 x 128
    entries (weights) instead of 128 of a row.  ``layout``: "rows" (codes [R, C]),
    "columns" (of x transposed: codes [C, R]) or "both" (a pair of the two, from
    one reading of x).  ``out``: an earlier result of the same shapes,
    overwritten."""
    if layout not in ("rows", "columns", "both"):
        raise ValueError("layout must be rows, columns or both")
    m, dev = _matrix(x, "x"), x.device
    R, C = x.shape
    shapes = ((R, C),) if layout == "rows" else ((C, R),) if layout == "columns" else ((R, C), (C, R))
    given = () if out is None else tuple(out) if layout == "both" else (out,)
    sp, on = _stream(dev, stream, (x, *(t for b in given for t in b[:2])) if stream is not None else ())
    if out is None:
        with on:
            given, made = zip(*(_new(*shape, square, dev) for shape in shapes))
    else:
        made = [_blocks(b, "out", dev) for b in given]
        for b, o, shape in zip(given, made, shapes):
            if (o.rows, o.cols) != shape or b.scales.shape[0] != (-(-shape[0] // TN_BLOCK8) if square else shape[0]):
                raise ValueError("out does not have the result's shapes")
            if not b.powers:
                raise ValueError("out is marked as having other scales than powers of two")
            o.block_rows = TN_BLOCK8 if square else 1
    st = _lib().tn_block8_quantize(m, made[0] if layout != "columns" else None,
                                   made[-1] if layout != "rows" else None, sp)
    if st:
        _check(st)
    return given if layout == "both" else given[0]


def _out(out, shape, dtype, device, on):
    dtype = dtype or (out.dtype if out is not None else _TORCH.bfloat16)
    if dtype not in _types():
        raise ValueError("dtype must be float32, bfloat16 or float16")
    if out is None:
        with on:
            return _TORCH.empty(shape, dtype=dtype, device=device)
    if tuple(out.shape) != shape or out.dtype is not dtype or out.device != device:
        raise ValueError(f"out must be a {dtype} tensor of shape {shape} on the operands' device")
    if out.is_neg() or (shape[1] > 1 and out.stride(1) != 1) or (shape[0] > 1 and out.stride(0) < shape[1]):
        raise ValueError("rows of out must be contiguous and not overlap")
    return out


def _product(a: tn_block8, b: tn_block8, out, sp):
    stride = out.stride(0) if out.shape[0] > 1 else max(1, out.shape[1])
    st = _lib().tn_block8_product(a, b, out.data_ptr(), _types()[out.dtype], stride, sp)
    if st:
        _check(st)


def product8(a: Blocks8, b: Blocks8, dtype=None, out=None, stream=None):
    """``a b^T`` ([m, n], ``dtype`` float32, bfloat16 (default) or float16) of quantised
    [m, k] and [n, k]."""
    _types()
    dev = a.codes.device
    if dev.type != "cuda" or dev.index != _TORCH._C._cuda_getDevice():
        raise ValueError(f"a is on {dev}, which is not the current device")
    A, B = _blocks(a, "a", dev), _blocks(b, "b", dev)
    sp, on = _stream(dev, stream, (*a[:2], *b[:2], out) if stream is not None else ())
    out = _out(out, (A.rows, B.rows), dtype, dev, on)
    _product(A, B, out, sp)
    return out


def linear8(x, w: Blocks8, dtype=None, out=None, stream=None):
    """``Q(x) w^T`` ([R, n], ``dtype`` that of x by default) of rows ``x`` [R, k], which
    are quantised on the way, and weights ``w`` [n, k]."""
    m, dev = _matrix(x, "x"), x.device
    W = _blocks(w, "w", dev)
    if W.cols != m.cols:
        raise ValueError(f"x has {m.cols} columns, w {W.cols}")
    sp, on = _stream(dev, stream, (x, *w[:2], out) if stream is not None else ())
    out = _out(out, (m.rows, W.rows), dtype or (out.dtype if out is not None else x.dtype), dev, on)
    with on:
        q = _Scratch(m.rows, m.cols, dev)
    st = _lib().tn_block8_quantize(m, q.blocks, None, sp)
    if st:
        _check(st)
    _product(q.blocks, W, out, sp)
    return out


def linear8_grad(x, dy, w: Blocks8, dtype=None, stream=None):
    """Gradients of ``linear8`` from ``dy`` [R, n]: (dx [R, k] of x's type, dW [n, k] of
    ``dtype``, float32 by default).  ``w`` is the transposed weight [k, n], as
    ``quantize8(weight, square=True, layout="columns")`` makes it.  dx = Q(dy) W;
    dW = Q'(dy)^T Q'(x) with x and dy quantised along their rows' number (which is
    taken as having no gradient of its own)."""
    X, Y, dev = _matrix(x, "x"), _matrix(dy, "dy"), x.device
    W = _blocks(w, "w", dev)
    R, k, n = X.rows, X.cols, Y.cols
    if dy.device != dev or Y.rows != R or W.rows != k or W.cols != n:
        raise ValueError(f"x must be [R, k], dy [R, n] and w the transposed weight [k, n] on one device, not "
                         f"{tuple(x.shape)}, {tuple(dy.shape)} and {tuple(w.codes.shape)}")
    sp, on = _stream(dev, stream, (x, dy, *w[:2]))
    dx = _out(None, (R, k), x.dtype, dev, on)
    dw = _out(None, (n, k), dtype or _F32, dev, on)
    with on:
        qy, qyt, qxt = _Scratch(R, n, dev), _Scratch(n, R, dev), _Scratch(k, R, dev)
    L = _lib()
    st = L.tn_block8_quantize(Y, qy.blocks, qyt.blocks, sp) or L.tn_block8_quantize(X, None, qxt.blocks, sp)
    if st:
        _check(st)
    _product(qy.blocks, W, dx, sp)
    _product(qyt.blocks, qxt.blocks, dw, sp)
    return dx, dw
