"""Python binding of the filtered distributions of libspecverify (``include/specsample.h``; argument marshalling only).

What a batch's requests ask for is a Filter; a draft model's tokens are drawn with it, and the verify step's rows
filtered alike:

    f = Filter(temperature, top_k, top_p, min_p)           # an entry a request
    f.sample(draft_logits, uniforms, tokens)               # one token a row
    f.mask(target_logits, out)                             # -inf where a token is not kept

Rows that share requests (a sequence's gamma + 1 rows) name them with ``request``. Masked rows keep their logits as they
are: a verify call has to be given the requests' temperature, which is one, or 0, for all that it verifies. Every call enqueues on the given
stream (default: torch's current one) and returns the library's host status code. The library reads tensors by
address: a Filter keeps references to its own, and a caller using another stream than the one its tensors were made
on orders the two itself.
"""
from __future__ import annotations

import ctypes

import torch

from .specverify import SV_BF16, SV_F32, _ptr, lib

SV_MAX_FILTER_V = 262144

# every exported symbol of specsample.h, in header order
EXPORTS = ("spec_filter", "spec_sample")


class SvFilter(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
                ("min_p", ctypes.c_void_p), ("request", ctypes.c_void_p), ("requests", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def _bind():
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.spec_filter.argtypes = [vp, ctypes.c_int, i32, i32, i64, vp, vp, i64, vp, vp, vp]
    lib.spec_filter.restype = ctypes.c_int
    lib.spec_sample.argtypes = [vp, ctypes.c_int, i32, i32, i64, vp, vp, vp, vp, vp, vp, vp]
    lib.spec_sample.restype = ctypes.c_int


_bind()


def _ref(s):
    return None if s is None else ctypes.addressof(s)


def spec_filter(logits, dtype, rows, V, stride, filter, out, out_stride, out_kept, device_status, cuda_stream) -> int:
    """Filtered logits. filter: SvFilter or None; the rest sizes and device addresses."""
    return lib.spec_filter(logits, dtype, rows, V, stride, _ref(filter), out, out_stride, out_kept, device_status, cuda_stream)


def spec_sample(logits, dtype, rows, V, stride, filter, uniforms, out_tokens, out_logprob, out_kept, device_status,
                cuda_stream) -> int:
    """One token a row. filter: SvFilter or None; the rest sizes and device addresses."""
    return lib.spec_sample(logits, dtype, rows, V, stride, _ref(filter), uniforms, out_tokens, out_logprob, out_kept,
                           device_status, cuda_stream)


_TYPES = {torch.bfloat16: SV_BF16, torch.float32: SV_F32}


class Filter:
    """What requests ask for: float32 temperature, top_p, min_p and int32 top_k, an entry a request, or None.

    request: int32, a row's entry (None: rows have their own). device: where the calls run, needed only if every
    argument is None. The object holds the calls' status word.
    """

    def __init__(self, temperature=None, top_k=None, top_p=None, min_p=None, request=None, device=None):
        given = [t for t in (temperature, top_k, top_p, min_p) if t is not None]
        if device is None:
            if not given and request is None:
                raise ValueError("a filter of nothing needs a device")
            device = (given + [request])[0].device
        requests = given[0].numel() if given else 2 ** 31 - 1
        at = torch.empty(0, device=device).get_device()
        for t, name, kind in ((temperature, "temperature", torch.float32), (top_k, "top_k", torch.int32),
                              (top_p, "top_p", torch.float32), (min_p, "min_p", torch.float32), (request, "request", torch.int32)):
            if t is None:
                continue
            if t.dtype != kind:
                raise TypeError(f"{name} must be {kind}, got {t.dtype}")
            if t.dim() != 1 or not t.is_contiguous() or (name != "request" and t.numel() != requests):
                raise ValueError(f"{name} must be contiguous, an entry a request, got {tuple(t.shape)}")
            if t.get_device() != at:
                raise ValueError(f"{name} must be on device {at}, got {t.device}")
        self.temperature, self.top_k, self.top_p, self.min_p, self.request = temperature, top_k, top_p, min_p, request
        self.requests, self._device = requests, at
        self.struct = SvFilter(_ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p), _ptr(request), requests, 0)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self._at, self._status = ctypes.addressof(self.struct), _ptr(self.status)

    def _rows(self, t, name):
        """Rows of logits: their number, columns and stride."""
        if t.dim() != 2 or t.get_device() != self._device:
            raise ValueError(f"{name} must be [rows, columns] on device {self._device}, got {tuple(t.shape)} on {t.device}")
        rows, V = t.shape
        s0, s1 = t.stride()
        if s1 != 1 and V > 1:
            raise ValueError(f"{name}'s rows must be contiguous")
        return rows, V, s0 if rows > 1 else max(V, 1)

    def _entries(self, t, name, rows, kind):
        if t.dtype != kind:
            raise TypeError(f"{name} must be {kind}, got {t.dtype}")
        if t.dim() != 1 or t.shape[0] != rows or not t.is_contiguous() or t.get_device() != self._device:
            raise ValueError(f"{name} must be contiguous, [{rows}], on device {self._device}, got {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def _code(self, t, rows):
        code = _TYPES.get(t.dtype)
        if code is None:
            raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")
        if self.request is not None:
            if self.request.shape[0] != rows:
                raise ValueError(f"request has {self.request.shape[0]} rows, the logits {rows}")
        elif rows > self.requests:
            raise ValueError(f"the filter has {self.requests} requests, the logits {rows} rows")
        return code

    def _stream(self, stream):
        if self._device < 0:
            raise ValueError("the filter's tensors must be on a CUDA device")
        if stream is not None:
            return stream.cuda_stream
        return torch._C._cuda_getCurrentRawStream(self._device)  # the current stream's handle alone

    def mask(self, logits, out, out_kept=None, stream=None) -> int:
        """Enqueue spec_filter: logits where a token is kept, -inf elsewhere. out may be logits itself."""
        rows, V, stride = self._rows(logits, "logits")
        code = self._code(logits, rows)
        if out.dtype != logits.dtype or out.shape != logits.shape:
            raise ValueError(f"out must be like logits, got {tuple(out.shape)} of {out.dtype}")
        out_stride = self._rows(out, "out")[2]
        kept = None if out_kept is None else self._entries(out_kept, "out_kept", rows, torch.int32)
        return lib.spec_filter(logits.data_ptr(), code, rows, V, stride, self._at, out.data_ptr(), out_stride, kept, self._status,
                               self._stream(stream))

    def sample(self, logits, uniforms, out_tokens, out_logprob=None, out_kept=None, stream=None) -> int:
        """Enqueue spec_sample: a token a row, drawn with uniforms (float32 in [0, 1))."""
        rows, V, stride = self._rows(logits, "logits")
        code = self._code(logits, rows)
        u = self._entries(uniforms, "uniforms", rows, torch.float32)
        tokens = self._entries(out_tokens, "out_tokens", rows, torch.int32)
        logprob = None if out_logprob is None else self._entries(out_logprob, "out_logprob", rows, torch.float32)
        kept = None if out_kept is None else self._entries(out_kept, "out_kept", rows, torch.int32)
        return lib.spec_sample(logits.data_ptr(), code, rows, V, stride, self._at, u, tokens, logprob, kept, self._status,
                               self._stream(stream))

    def status_bits(self) -> int:
        return int(self.status.item()) & 0xFFFFFFFF
