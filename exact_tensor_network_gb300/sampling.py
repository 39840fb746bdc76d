"""Outcomes drawn from rows by given random numbers (``include/tn_sampling.h``).

The functions carry the C names and only marshal arguments; ``Sampler`` is a small
class over torch tensors.  Rows are those of ``Outcomes``: amplitudes (complex64,
as ``Plan.execute`` writes them) or real logits (float32, bfloat16, float16).
Every call runs in the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

from .outcomes import _types, tn_rows

_P = ctypes.c_void_p
_I32, _I64, _F32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class tn_filters(ctypes.Structure):
    _fields_ = [("temperature", _F32), ("top_p", _F32), ("min_p", _F32), ("top_k", _I32),
                ("temperatures", _P), ("top_ps", _P), ("min_ps", _P), ("top_ks", _P)]


_RP, _FP = ctypes.POINTER(tn_rows), ctypes.POINTER(tn_filters)

# exported symbol -> (restype, argtypes)
SIGNATURES = {
    "tn_sampler_create": (ctypes.c_int, [_I32, _I64, _I64, _F32, ctypes.POINTER(_P)]),
    "tn_sampler_destroy": (None, [_P]),
    "tn_sampler_workspace_bytes": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_uint64)]),
    "tn_sampler_set_workspace": (ctypes.c_int, [_P, _P, ctypes.c_uint64]),
    "tn_sampler_draw": (ctypes.c_int, [_P, _RP, _FP, _P, _I32, _I64, _P, _P, _P, _P]),
    "tn_sampler_check": (ctypes.c_int, [_P]),
    "tn_sampler_last_error": (ctypes.c_char_p, [_P]),
}


def _lib():
    from . import lib
    return lib()


def _check(st: int, handle=None) -> None:
    if st != 0:
        from . import TNError, tn_status_string
        msg = _lib().tn_sampler_last_error(handle)
        raise TNError(st, (msg.decode() if msg else "") or tn_status_string(st))


# ---- functions with the C names -------------------------------------------

def tn_sampler_create(type_: int, cols: int, max_rows: int, scale: float) -> int:
    """Make a handle (an integer) for rows of ``cols`` entries."""
    out = _P()
    _check(_lib().tn_sampler_create(type_, cols, max_rows, scale, ctypes.byref(out)))
    return out.value


def tn_sampler_destroy(handle: int) -> None:
    _lib().tn_sampler_destroy(handle)


def tn_sampler_workspace_bytes(handle: int) -> int:
    v = ctypes.c_uint64()
    _check(_lib().tn_sampler_workspace_bytes(handle, ctypes.byref(v)), handle)
    return v.value


def tn_sampler_set_workspace(handle: int, dev_ptr: int, nbytes: int) -> None:
    _check(_lib().tn_sampler_set_workspace(handle, dev_ptr, nbytes), handle)


def tn_sampler_draw(handle: int, rows: tn_rows, filters: tn_filters, u: int, wide: int, draws: int, ids: int,
                    logp: int, kept: int, stream: int = 0) -> None:
    _check(_lib().tn_sampler_draw(handle, rows, filters, u, wide, draws, ids, logp, kept, stream), handle)


def tn_sampler_check(handle: int) -> None:
    _check(_lib().tn_sampler_check(handle), handle)


def tn_sampler_last_error(handle: Optional[int] = None) -> str:
    return _lib().tn_sampler_last_error(handle).decode()


# ---- convenience wrapper over torch tensors --------------------------------

class Samples(NamedTuple):
    """``Sampler.sample``: outcomes [R, draws], their log probabilities among the
    entries left, and the number of those [R]."""
    ids: object
    logp: object
    kept: object


class Sampler:
    """Owns a handle and (optionally) a torch workspace tensor.

    ``cols`` entries a row of ``dtype`` (complex64 amplitudes, or float32,
    bfloat16 or float16 logits), at most ``max_rows`` rows a call and ``draws`` draws
    of each (None: any number), inverse temperature ``scale`` before any other.

    Rows and masks are those of ``Outcomes``.  All tensors of a call, its
    stream and the workspace are on the current device; the first call binds a
    workspace there unless ``bind_workspace`` did, and waits for the device once
    (so bind it before a call is captured into a graph, which works in it: keep the
    sampler, and bind no other, as long as the graph).

    Calls are asynchronous on ``stream`` (default: torch's current stream).
    On another stream the caller orders it after the inputs' producers; outputs
    made by the call belong to that stream, and the inputs, ``out`` and the
    workspace are recorded on it.
    """

    def __init__(self, cols: int, dtype=None, max_rows: int = 1, scale: float = 1.0, draws: Optional[int] = None):
        import torch
        self.handle = None
        dtype = torch.complex64 if dtype is None else dtype
        if dtype not in _types():
            raise ValueError("dtype must be complex64, float32, bfloat16 or float16")
        if draws is not None and (draws != int(draws) or draws < 0):
            raise ValueError("draws must be None or a whole number >= 0")
        self.draws = None if draws is None else int(draws)
        self.handle = tn_sampler_create(_types()[dtype], int(cols), int(max_rows), float(scale))
        self.cols, self.dtype, self.max_rows, self.scale = int(cols), dtype, int(max_rows), float(scale)
        self._ws, self._ws_streams = None, set()
        self._index = None          # of the workspace's device
        # looked up once: small calls cost what their host side costs
        self._torch, self._L = torch, _lib()
        self._current_device = torch._C._cuda_getDevice
        self._empty, self._i64, self._f32 = torch.empty, torch.int64, torch.float32
        self._r, self._f = tn_rows(), tn_filters()
        self._rp, self._fp = ctypes.byref(self._r), ctypes.byref(self._f)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            try:
                tn_sampler_destroy(h)
            except Exception:      # interpreter shutdown
                pass
            self.handle = None

    workspace_bytes = property(lambda self: tn_sampler_workspace_bytes(self.handle))

    def bind_workspace(self, device=None):
        """Allocate the workspace with torch on ``device`` (default: the
        current one) and bind it.  Waits for the device."""
        torch = self._torch
        nbytes = self.workspace_bytes
        device = torch.device("cuda" if device is None else device)
        with torch.cuda.device(device):
            ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
            tn_sampler_set_workspace(self.handle, (ws.data_ptr() + 255) // 256 * 256, nbytes)
        self._ws, self._ws_streams, self._index = ws, set(), ws.device.index
        return ws

    def _parameter(self, value, off, name, dtype, R, device):
        """(one number for all rows, pointer to each row's or None)."""
        if value is None:
            return off, None
        if isinstance(value, self._torch.Tensor):
            if value.dtype is not dtype or value.device != device or value.numel() != R or not value.is_contiguous():
                raise ValueError(f"{name} must be a number or a contiguous {dtype} tensor of {R} entries on the "
                                 "rows' device")
            return off, value.data_ptr()
        return value, None

    def _use_workspace(self, stream):
        # freed with the handle, it must outlive the work on every stream
        self._ws.record_stream(stream)
        self._ws_streams.add(stream.cuda_stream)

    def _new(self, R, shape, device):
        empty = self._empty
        return Samples(empty(shape, dtype=self._i64, device=device), empty(shape, dtype=self._f32, device=device),
                       empty(R, dtype=self._i64, device=device))

    def sample(self, rows, u, temperature=None, top_k=None, top_p=None, min_p=None, mask=None,
               out: Optional[Samples] = None, stream=None) -> Samples:
        """Draw outcomes of every row ([R, cols] or [cols]) with the random numbers
        ``u`` ([R, draws], or [R] for one draw each, float32 or float64 in [0, 1)).
        ``temperature``, ``top_p``, ``min_p`` (float32) and ``top_k`` (int32) are a
        number for all rows or a tensor [R]; None is no filter.  ``out``: an
        earlier result of the same shapes, overwritten."""
        torch = self._torch
        if rows.dim() == 1:
            rows = rows.unsqueeze(0)
        shape = rows.shape
        if len(shape) != 2 or shape[1] != self.cols:
            raise ValueError(f"rows must be [R, {self.cols}], not {tuple(shape)}")
        if rows.dtype is not self.dtype or not rows.is_cuda:
            raise ValueError(f"rows must be {self.dtype} CUDA tensors")
        if rows.is_conj() or rows.is_neg():
            raise ValueError("rows are a lazily conjugated or negated view: resolve it first")
        R, device, s, f = shape[0], rows.device, self._r, self._f
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
            if mask.dtype not in (torch.bool, torch.uint8) or mask.device != device:
                raise ValueError("mask must be a bool or uint8 tensor on the rows' device")
            mask = mask.expand(R, self.cols)
            s.mask = mask.data_ptr()
            s.mask_row_stride, s.mask_col_stride = mask.stride()
        if u.dtype is torch.float32:
            wide = 0
        elif u.dtype is torch.float64:
            wide = 1
        else:
            raise ValueError("u must be float32 or float64")
        ushape = u.shape
        if not 1 <= len(ushape) <= 2 or ushape[0] != R or u.device != device or not u.is_contiguous():
            raise ValueError(f"u must be a contiguous tensor [{R}] or [{R}, draws] on the rows' device")
        draws = ushape[1] if len(ushape) == 2 else 1
        if self.draws is not None and draws > self.draws:
            raise ValueError(f"{draws} draws of a row: the sampler was made for at most {self.draws}")
        f.temperature, f.temperatures = self._parameter(temperature, 1.0, "temperature", self._f32, R, device)
        if isinstance(top_k, int):
            top_k = max(0, min(top_k, self.cols))       # (a larger number would wrap around)
        f.top_k, f.top_ks = self._parameter(top_k, 0, "top_k", torch.int32, R, device)
        f.top_p, f.top_ps = self._parameter(top_p, 1.0, "top_p", self._f32, R, device)
        f.min_p, f.min_ps = self._parameter(min_p, 0.0, "min_p", self._f32, R, device)
        if stream is None:
            sp = torch._C._cuda_getCurrentRawStream(index)
            if sp not in self._ws_streams:
                self._use_workspace(torch.cuda.current_stream(device))
            if out is None:
                out = self._new(R, ushape, device)
        else:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            elif getattr(stream, "device", device) != device:
                raise ValueError(f"the stream is on {stream.device}, the rows on {device}")
            for t in (rows, u, mask, temperature, top_k, top_p, min_p, *(out or ())):
                if isinstance(t, torch.Tensor):
                    t.record_stream(stream)
            sp = stream.cuda_stream
            if sp not in self._ws_streams:
                self._use_workspace(stream)
            if out is None:
                with torch.cuda.stream(stream):
                    out = self._new(R, ushape, device)
        for t, n, dtype, name in ((out.ids, R * draws, self._i64, "ids"), (out.logp, R * draws, self._f32, "logp"),
                                  (out.kept, R, self._i64, "kept")):
            if t.dtype is not dtype or t.device != device or t.numel() != n or not t.is_contiguous():
                raise ValueError(f"out.{name} must be a contiguous {dtype} tensor of {n} entries on the rows' device")
        st = self._L.tn_sampler_draw(self.handle, self._rp, self._fp, u.data_ptr(), wide, draws, out.ids.data_ptr(),
                                     out.logp.data_ptr(), out.kept.data_ptr(), sp)
        if st:
            _check(st, self.handle)
        return out

    def check(self) -> None:
        """After a synchronise: raises if a call met an invalid parameter or random number."""
        tn_sampler_check(self.handle)
