"""Operators on outcome distributions (``include/tn_outcomes.h``).

The functions carry the C names and only marshal arguments; ``Outcomes`` is a
small class over torch tensors.  Rows are amplitudes (complex64, as
``Plan.execute`` writes them) or real logits (float32, bfloat16, float16);
definitions of absent entries, empty rows, ties and invalid ids are those of
the header.  Every call runs in the library's CUDA kernels; there is no
fallback.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

_P = ctypes.c_void_p
_I32, _I64, _F32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float

# entry types
TN_TYPE_C64, TN_TYPE_F32, TN_TYPE_BF16, TN_TYPE_F16 = 0, 1, 2, 3
TN_OUTCOMES_MAX_TOP = 128
TN_OUTCOMES_MAX_IDS = 256


class tn_rows(ctypes.Structure):
    _fields_ = [("data", _P), ("rows", _I64), ("row_stride", _I64), ("col_stride", _I64),
                ("mask", _P), ("mask_row_stride", _I64), ("mask_col_stride", _I64)]


class tn_teacher(ctypes.Structure):
    _fields_ = [("ids", _P), ("logits", _P), ("type", _I32), ("count", _I32), ("scale", _F32)]


_RP, _TP = ctypes.POINTER(tn_rows), ctypes.POINTER(tn_teacher)

# exported symbol -> (restype, argtypes)
SIGNATURES = {
    "tn_outcomes_create": (ctypes.c_int, [_I32, _I64, _I64, _I32, _F32, ctypes.POINTER(_P)]),
    "tn_outcomes_destroy": (None, [_P]),
    "tn_outcomes_workspace_bytes": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_uint64)]),
    "tn_outcomes_set_workspace": (ctypes.c_int, [_P, _P, ctypes.c_uint64]),
    "tn_outcomes_score": (ctypes.c_int, [_P, _RP, _P, _I32, _P, _P, _P, _I32, _P, _P, _P]),
    "tn_outcomes_score_grad": (ctypes.c_int, [_P, _RP, _P, _I32, _P, _P, _P, _P, _P, _I64, _I64, _P]),
    "tn_outcomes_distill": (ctypes.c_int, [_P, _RP, _TP, _P, _P, _P]),
    "tn_outcomes_distill_grad": (ctypes.c_int, [_P, _RP, _TP, _P, _P, _P, _I64, _I64, _P]),
    "tn_outcomes_distill_step": (ctypes.c_int, [_P, _RP, _TP, _P, _P, _P, _P, _I64, _I64, _P]),
    "tn_outcomes_check": (ctypes.c_int, [_P]),
    "tn_outcomes_last_error": (ctypes.c_char_p, [_P]),
}


def _lib():
    from . import lib
    return lib()


def _check(st: int, handle=None) -> None:
    if st != 0:
        from . import TNError, tn_status_string
        msg = _lib().tn_outcomes_last_error(handle)
        raise TNError(st, (msg.decode() if msg else "") or tn_status_string(st))


# ---- functions with the C names -------------------------------------------

def tn_outcomes_create(type_: int, cols: int, max_rows: int, max_top: int, scale: float) -> int:
    """Make a handle (an integer) for rows of ``cols`` entries."""
    out = _P()
    _check(_lib().tn_outcomes_create(type_, cols, max_rows, max_top, scale, ctypes.byref(out)))
    return out.value


def tn_outcomes_destroy(handle: int) -> None:
    _lib().tn_outcomes_destroy(handle)


def tn_outcomes_workspace_bytes(handle: int) -> int:
    v = ctypes.c_uint64()
    _check(_lib().tn_outcomes_workspace_bytes(handle, ctypes.byref(v)), handle)
    return v.value


def tn_outcomes_set_workspace(handle: int, dev_ptr: int, nbytes: int) -> None:
    _check(_lib().tn_outcomes_set_workspace(handle, dev_ptr, nbytes), handle)


def tn_outcomes_score(handle: int, rows: tn_rows, given: int, n_given: int, logp: int, logz: int,
                      entropy: int, n_top: int, top_ids: int, top_logp: int, stream: int = 0) -> None:
    _check(_lib().tn_outcomes_score(handle, rows, given, n_given, logp, logz, entropy, n_top, top_ids,
                                    top_logp, stream), handle)


def tn_outcomes_score_grad(handle: int, rows: tn_rows, given: int, n_given: int, logz: int,
                           entropy: int, g_logp: int, g_entropy: int, grad: int, grad_row_stride: int,
                           grad_col_stride: int, stream: int = 0) -> None:
    _check(_lib().tn_outcomes_score_grad(handle, rows, given, n_given, logz, entropy, g_logp, g_entropy,
                                         grad, grad_row_stride, grad_col_stride, stream), handle)


def tn_outcomes_distill(handle: int, rows: tn_rows, teacher: tn_teacher, loss: int, logz: int,
                        stream: int = 0) -> None:
    _check(_lib().tn_outcomes_distill(handle, rows, teacher, loss, logz, stream), handle)


def tn_outcomes_distill_grad(handle: int, rows: tn_rows, teacher: tn_teacher, logz: int, g_loss: int,
                             grad: int, grad_row_stride: int, grad_col_stride: int,
                             stream: int = 0) -> None:
    _check(_lib().tn_outcomes_distill_grad(handle, rows, teacher, logz, g_loss, grad, grad_row_stride,
                                           grad_col_stride, stream), handle)


def tn_outcomes_distill_step(handle: int, rows: tn_rows, teacher: tn_teacher, g_loss: int, loss: int,
                             logz: int, grad: int, grad_row_stride: int, grad_col_stride: int,
                             stream: int = 0) -> None:
    _check(_lib().tn_outcomes_distill_step(handle, rows, teacher, g_loss, loss, logz, grad,
                                           grad_row_stride, grad_col_stride, stream), handle)


def tn_outcomes_check(handle: int) -> None:
    _check(_lib().tn_outcomes_check(handle), handle)


def tn_outcomes_last_error(handle: Optional[int] = None) -> str:
    return _lib().tn_outcomes_last_error(handle).decode()


# ---- convenience wrapper over torch tensors --------------------------------

class Scores(NamedTuple):
    """``Outcomes.score``: log Z, entropy, log p of the given outcomes (None
    without any) and the alternatives (None with ``top=0``)."""
    logz: object
    entropy: object
    logp: object
    top_ids: object
    top_logp: object


class Distill(NamedTuple):
    """``Outcomes.distill`` and ``distill_step`` (``grad`` only there)."""
    loss: object
    logz: object
    grad: object = None


_TYPES = None   # torch dtype -> TN_TYPE_*, filled on first use (torch is imported late)


def _types():
    global _TYPES
    if _TYPES is None:
        import torch
        _TYPES = {torch.complex64: TN_TYPE_C64, torch.float32: TN_TYPE_F32,
                  torch.bfloat16: TN_TYPE_BF16, torch.float16: TN_TYPE_F16}
    return _TYPES


class Outcomes:
    """Owns a handle and (optionally) a torch workspace tensor.

    ``cols`` entries a row of ``dtype`` (complex64 amplitudes, or float32,
    bfloat16 or float16 logits), at most ``max_rows`` rows a call, ``top``
    alternatives, inverse temperature ``scale``.

    Rows are CUDA tensors ``[R, cols]`` of any strides (innermost 1 is the
    fast layout) or ``[cols]`` (one row).  ``mask`` is a bool or uint8 tensor
    that broadcasts to the rows (0 = absent).  Ids are int64.  All tensors of
    a call, its stream and the workspace are on the current device; the first
    call binds a workspace there unless ``bind_workspace`` did, and waits for
    the device once (so bind it before a call is captured into a graph).

    Calls are asynchronous on ``stream`` (default: torch's current stream).
    On another stream the caller orders it after the inputs' producers, as for
    any other launch; outputs made by the call belong to that stream, and the
    inputs, ``out`` and the workspace are recorded on it.  ``out`` of a gradient
    may not overlap the rows.
    """

    def __init__(self, cols: int, dtype=None, max_rows: int = 1, top: int = 0, scale: float = 1.0):
        import torch
        self.handle = None
        dtype = torch.complex64 if dtype is None else dtype
        if dtype not in _types():
            raise ValueError("dtype must be complex64, float32, bfloat16 or float16")
        self.handle = tn_outcomes_create(_types()[dtype], int(cols), int(max_rows), int(top), float(scale))
        self.cols, self.dtype, self.max_rows = int(cols), dtype, int(max_rows)
        self.top, self.scale = int(top), float(scale)
        self._ws, self._ws_streams = None, set()
        self._index = None          # of the workspace's device
        # the small calls cost what their host side costs: what does not
        # change from call to call is looked up once
        self._torch, self._L = torch, _lib()
        self._current_device = torch._C._cuda_getDevice
        self._empty, self._f32, self._teacher_types = torch.empty, torch.float32, _types()
        self._r, self._t = tn_rows(), tn_teacher()
        self._rp, self._tp = ctypes.byref(self._r), ctypes.byref(self._t)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            try:
                tn_outcomes_destroy(h)
            except Exception:      # interpreter shutdown
                pass
            self.handle = None

    workspace_bytes = property(lambda self: tn_outcomes_workspace_bytes(self.handle))

    def bind_workspace(self, device=None):
        """Allocate the workspace with torch on ``device`` (default: the
        current one) and bind it.  Waits for the device."""
        import torch
        nbytes = self.workspace_bytes
        device = torch.device("cuda" if device is None else device)
        with torch.cuda.device(device):     # the library clears it on the current device
            ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
            tn_outcomes_set_workspace(self.handle, (ws.data_ptr() + 255) // 256 * 256, nbytes)
        self._ws, self._ws_streams, self._index = ws, set(), ws.device.index
        return ws

    # -- arguments --

    def _rows(self, rows, mask):
        """Check the rows and the mask into self._r; (rows, device, R)."""
        if rows.dim() == 1:
            rows = rows.unsqueeze(0)
        shape = rows.shape
        if len(shape) != 2 or shape[1] != self.cols:
            raise ValueError(f"rows must be [R, {self.cols}], not {tuple(shape)}")
        if rows.dtype is not self.dtype or not rows.is_cuda:
            raise ValueError(f"rows must be {self.dtype} CUDA tensors")
        if rows.is_conj() or rows.is_neg():
            raise ValueError("rows are a lazily conjugated or negated view: resolve it first")
        R, device, s = shape[0], rows.device, self._r
        # kernels go to the current device, with the workspace's addresses
        index = device.index
        if index != self._current_device():
            raise ValueError(f"rows are on {device}, which is not the current device")
        if self._ws is None:
            self.bind_workspace(device)
        elif index != self._index:
            raise ValueError(f"rows are on {device}, the workspace is on cuda:{self._index}")
        s.data, s.rows = rows.data_ptr(), R
        s.row_stride, s.col_stride = rows.stride()
        if mask is None:
            s.mask = None
        else:
            torch = self._torch
            if mask.dtype not in (torch.bool, torch.uint8) or mask.device != device:
                raise ValueError("mask must be a bool or uint8 tensor on the rows' device")
            mask = mask.expand(R, self.cols)
            s.mask = mask.data_ptr()
            s.mask_row_stride, s.mask_col_stride = mask.stride()
        return rows, device, R

    def _on(self, device, stream, inputs):
        """(stream handle, torch stream to allocate outputs on or None)."""
        torch = self._torch
        if stream is None:
            raw = torch._C._cuda_getCurrentRawStream(device.index)
            if raw not in self._ws_streams:
                self._use_workspace(torch.cuda.current_stream(device))
            return raw, None
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        elif getattr(stream, "device", device) != device:
            raise ValueError(f"the stream is on {stream.device}, the rows on {device}")
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
        if stream.cuda_stream not in self._ws_streams:
            self._use_workspace(stream)
        return stream.cuda_stream, stream

    def _use_workspace(self, stream):
        # freed with the handle, it must outlive the work on every stream
        self._ws.record_stream(stream)
        self._ws_streams.add(stream.cuda_stream)

    def _vec(self, t, n, name, device, dtype=None):
        dtype = dtype or self._f32
        if t.dtype is not dtype or t.device != device or t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} entries on the rows' device")
        return t.data_ptr()

    def _ids(self, ids, R, name, device):
        if ids.dtype is not self._torch.int64 or ids.device != device or not ids.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int64 tensor on the rows' device")
        shape = ids.shape
        if not 1 <= len(shape) <= 2 or shape[0] != R:
            raise ValueError(f"{name} must be [{R}] or [{R}, n], not {tuple(shape)}")
        return shape[1] if len(shape) == 2 else 1

    def _teacher(self, ids, logits, R, device, scale):
        """Check the teacher into self._t."""
        n = self._ids(ids, R, "ids", device)
        t = self._teacher_types.get(logits.dtype, TN_TYPE_C64)
        if (t == TN_TYPE_C64 or logits.shape != ids.shape or logits.device != device
                or not logits.is_contiguous()):
            raise ValueError("the teacher's logits must be a contiguous float32, bfloat16 or float16 "
                             "tensor of the ids' shape on the rows' device")
        s = self._t
        s.ids, s.logits, s.type, s.count, s.scale = ids.data_ptr(), logits.data_ptr(), t, n, scale

    def _grad(self, rows, R, out, device, stream):
        if out is None:
            if stream is None:
                return self._empty((R, self.cols), dtype=self.dtype, device=device)
            with self._torch.cuda.stream(stream):
                return self._empty((R, self.cols), dtype=self.dtype, device=device)
        if out.shape != rows.shape or out.dtype is not self.dtype or out.device != device:
            raise ValueError("out must have the rows' shape, type and device")
        if out.is_conj() or out.is_neg():
            raise ValueError("out is a lazily conjugated or negated view")
        return out

    # -- calls --

    def score(self, rows, given=None, mask=None, out: Optional[Scores] = None, stream=None) -> Scores:
        """Log Z, entropy, log probabilities of the ``given`` outcomes ([R] or
        [R, n] int64, -1 = none) and the ``top`` most likely outcomes of every
        row.  ``out``: an earlier result of the same shapes, overwritten."""
        rows, dev, R = self._rows(rows, mask)
        n, k = 0, self.top
        if given is not None:
            n = self._ids(given, R, "given", dev)
        sp, on = self._on(dev, stream, (rows, mask, given, *(out or ())) if stream is not None else ())
        logp = ids = lp = None
        if out is None:
            if on is None:
                out = self._new_scores(R, k, given, dev)
            else:
                with self._torch.cuda.stream(on):
                    out = self._new_scores(R, k, given, dev)
            logz, entropy = out[0].data_ptr(), out[1].data_ptr()
            if n:
                logp = out[2].data_ptr()
            if k:
                ids, lp = out[3].data_ptr(), out[4].data_ptr()
        else:
            logz = self._vec(out.logz, R, "out.logz", dev)
            entropy = self._vec(out.entropy, R, "out.entropy", dev)
            if n:
                logp = self._vec(out.logp, R * n, "out.logp", dev)
            if k:
                ids = self._vec(out.top_ids, R * k, "out.top_ids", dev, self._torch.int64)
                lp = self._vec(out.top_logp, R * k, "out.top_logp", dev)
        st = self._L.tn_outcomes_score(self.handle, self._rp, given.data_ptr() if n else None, n, logp,
                                       logz, entropy, k, ids, lp, sp)
        if st:
            _check(st, self.handle)
        return out

    def _new_scores(self, R, k, given, dev):
        empty, f32 = self._empty, self._f32
        return Scores(empty(R, dtype=f32, device=dev), empty(R, dtype=f32, device=dev),
                      None if given is None else empty(given.shape, dtype=f32, device=dev),
                      empty((R, k), dtype=self._torch.int64, device=dev) if k else None,
                      empty((R, k), dtype=f32, device=dev) if k else None)

    def score_grad(self, rows, given, logz, entropy, g_logp, g_entropy=None, mask=None, out=None,
                   stream=None):
        """Gradient of the rows from those of ``score``'s logp (``g_logp``, the
        shape of ``given``) and entropy (``g_entropy``, [R] or None).  For
        amplitudes dL/dRe + i dL/dIm, torch's convention."""
        rows, dev, R = self._rows(rows, mask)
        n, ids, gl, h, e = 0, None, None, None, None
        if given is not None:
            n = self._ids(given, R, "given", dev)
            gl = self._vec(g_logp, R * n, "g_logp", dev)
            ids = given.data_ptr()
        z = self._vec(logz, R, "logz", dev)
        if g_entropy is not None:
            h = self._vec(g_entropy, R, "g_entropy", dev)
            e = self._vec(entropy, R, "entropy", dev)
        sp, on = self._on(dev, stream, (rows, mask, given, logz, entropy, g_logp, g_entropy, out)
                          if stream is not None else ())
        g = self._grad(rows, R, out, dev, on)
        rs, cs = g.stride()
        st = self._L.tn_outcomes_score_grad(self.handle, self._rp, ids, n, z, e, gl, h, g.data_ptr(), rs,
                                            cs, sp)
        if st:
            _check(st, self.handle)
        return g

    def _new_loss(self, R, dev, stream):
        if stream is not None:
            with self._torch.cuda.stream(stream):
                return self._new_loss(R, dev, None)
        empty, f32 = self._empty, self._f32
        return empty(R, dtype=f32, device=dev), empty(R, dtype=f32, device=dev)

    def distill(self, rows, ids, logits, mask=None, teacher_scale: float = 1.0, stream=None) -> Distill:
        """Distance (KL) of every row from the teacher that gives its outcomes
        ``ids`` ([R, K] int64, -1 = none) the logits ``logits``."""
        rows, dev, R = self._rows(rows, mask)
        self._teacher(ids, logits, R, dev, teacher_scale)
        sp, on = self._on(dev, stream, (rows, mask, ids, logits) if stream is not None else ())
        loss, logz = self._new_loss(R, dev, on)
        st = self._L.tn_outcomes_distill(self.handle, self._rp, self._tp, loss.data_ptr(), logz.data_ptr(), sp)
        if st:
            _check(st, self.handle)
        return Distill(loss, logz)

    def distill_grad(self, rows, ids, logits, logz, g_loss, mask=None, teacher_scale: float = 1.0,
                     out=None, stream=None):
        """Gradient of the rows from that of ``distill``'s loss ([R])."""
        rows, dev, R = self._rows(rows, mask)
        self._teacher(ids, logits, R, dev, teacher_scale)
        z, w = self._vec(logz, R, "logz", dev), self._vec(g_loss, R, "g_loss", dev)
        sp, on = self._on(dev, stream, (rows, mask, ids, logits, logz, g_loss, out)
                          if stream is not None else ())
        g = self._grad(rows, R, out, dev, on)
        rs, cs = g.stride()
        st = self._L.tn_outcomes_distill_grad(self.handle, self._rp, self._tp, z, w, g.data_ptr(), rs, cs, sp)
        if st:
            _check(st, self.handle)
        return g

    def distill_step(self, rows, ids, logits, g_loss, mask=None, teacher_scale: float = 1.0, out=None,
                     stream=None) -> Distill:
        """Loss and gradient together, for a loss gradient ``g_loss`` ([R])
        that is known beforehand (1 / R for a mean over the rows)."""
        rows, dev, R = self._rows(rows, mask)
        self._teacher(ids, logits, R, dev, teacher_scale)
        w = self._vec(g_loss, R, "g_loss", dev)
        sp, on = self._on(dev, stream, (rows, mask, ids, logits, g_loss, out)
                          if stream is not None else ())
        loss, logz = self._new_loss(R, dev, on)
        g = self._grad(rows, R, out, dev, on)
        rs, cs = g.stride()
        st = self._L.tn_outcomes_distill_step(self.handle, self._rp, self._tp, w, loss.data_ptr(),
                                              logz.data_ptr(), g.data_ptr(), rs, cs, sp)
        if st:
            _check(st, self.handle)
        return Distill(loss, logz, g)

    def check(self) -> None:
        """After a synchronise: raises if a call met an id outside [-1, cols)."""
        tn_outcomes_check(self.handle)
