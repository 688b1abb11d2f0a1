"""Python binding of the cache calls of libspecverify (``include/speccache.h``; argument marshalling only).

A verify step's target model appends each chunk's keys and values to a paged cache, attends over it, and,
once a token tree is verified, keeps the accepted path:

    cache = PagedCache(k, v, page_table)             # k, v: [layers, pages, page_size, heads, head_dim]
    chunk = Chunk(seq_offsets, cached, rows, max_gamma, parents)
    for layer in range(layers):
        cache.append(chunk, q, k_new, v_new, q_rot, rope=rope, layer=layer)
        cache.attend(chunk, q_rot, out, scale=scale, layer=layer)
    ... logits, specverify.spec_verify_tree ...
    cache.compact(chunk, out_num_accepted, out_path, cached)

Every call enqueues on the given stream (default: torch's current one) and returns the library's host status
code. The library reads tensors by address: each object keeps references to the tensors it describes, and a
caller using another stream than the one its tensors were made on orders the two itself.
"""
from __future__ import annotations

import ctypes

import torch

from .specverify import SV_BF16, _ptr, lib

SV_F16, SV_E4M3 = 2, 3

# every exported symbol of speccache.h, in header order
EXPORTS = ("spec_cache_append", "spec_cache_workspace_size", "spec_cache_attend", "spec_cache_attend_ex",
           "spec_cache_compact")


class SvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("stride_page", ctypes.c_int64),
                ("stride_token", ctypes.c_int64), ("stride_head", ctypes.c_int64), ("stride_layer", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("layers", ctypes.c_int32), ("pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("table_stride", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class SvChunk(ctypes.Structure):
    _fields_ = [("seq_offsets", ctypes.c_void_p), ("cached", ctypes.c_void_p), ("parents", ctypes.c_void_p),
                ("B", ctypes.c_int32), ("rows", ctypes.c_int32), ("max_gamma", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class SvRope(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def _bind():
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.spec_cache_append.argtypes = [vp, i32, vp, vp, ctypes.c_int, i32, vp, i64, vp, vp, i64, vp, vp, vp]
    lib.spec_cache_append.restype = ctypes.c_int
    lib.spec_cache_workspace_size.argtypes = [vp]
    lib.spec_cache_workspace_size.restype = sz
    lib.spec_cache_attend.argtypes = [vp, i32, vp, ctypes.c_int, i32, vp, i64, ctypes.c_float, i32, vp, vp, vp, vp, sz,
                                      vp]
    lib.spec_cache_attend.restype = ctypes.c_int
    lib.spec_cache_attend_ex.argtypes = lib.spec_cache_attend.argtypes[:-1] + [vp, vp]
    lib.spec_cache_attend_ex.restype = ctypes.c_int
    lib.spec_cache_compact.argtypes = [vp, vp, vp, vp, vp, vp, vp]
    lib.spec_cache_compact.restype = ctypes.c_int


_bind()


def _ref(s):
    return None if s is None else ctypes.addressof(s)


def spec_cache_append(cache, layer, chunk, rope, dtype, q_heads, q, q_stride, k, v, kv_stride, q_out, device_status,
                      cuda_stream) -> int:
    """Rotate and append a chunk. cache, chunk, rope: SvCache, SvChunk, SvRope or None; the rest addresses."""
    return lib.spec_cache_append(_ref(cache), layer, _ref(chunk), _ref(rope), dtype, q_heads, q, q_stride, k, v,
                                 kv_stride, q_out, device_status, cuda_stream)


def spec_cache_workspace_size(cache) -> int:
    return lib.spec_cache_workspace_size(_ref(cache))


def spec_cache_attend(cache, layer, chunk, dtype, q_heads, q, q_stride, scale, window, out, lse, device_status,
                      workspace, workspace_bytes, cuda_stream) -> int:
    """Attention of a chunk over the cache. cache, chunk: SvCache, SvChunk or None; the rest addresses."""
    return lib.spec_cache_attend(_ref(cache), layer, _ref(chunk), dtype, q_heads, q, q_stride, scale, window, out, lse,
                                 device_status, workspace, workspace_bytes, cuda_stream)


def spec_cache_attend_ex(cache, layer, chunk, dtype, q_heads, q, q_stride, scale, window, out, lse, device_status,
                         workspace, workspace_bytes, debug, cuda_stream) -> int:
    """spec_cache_attend with the debug structure (specverify.SvDebug or None; spin_limit alone is read)."""
    return lib.spec_cache_attend_ex(_ref(cache), layer, _ref(chunk), dtype, q_heads, q, q_stride, scale, window, out,
                                    lse, device_status, workspace, workspace_bytes, _ref(debug), cuda_stream)


def spec_cache_compact(cache, chunk, out_num_accepted, out_path, out_cached, device_status, cuda_stream) -> int:
    """Keep the accepted path of a verified chunk. cache, chunk: SvCache, SvChunk or None; the rest addresses."""
    return lib.spec_cache_compact(_ref(cache), _ref(chunk), out_num_accepted, out_path, out_cached, device_status,
                                  cuda_stream)


# ------------------------------------------------------------------------------------------------
# torch marshalling helpers
# ------------------------------------------------------------------------------------------------
_ACTIVATIONS = {torch.bfloat16: SV_BF16, torch.float16: SV_F16}
_CACHES = {**_ACTIVATIONS, torch.float8_e4m3fn: SV_E4M3}


def _check(t, name, dtypes, shape=None, device=None):
    """A tensor argument's type, shape (None: any extent) and device number."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if shape is not None:
        got = t.shape
        if len(got) != len(shape) or any(w is not None and w != g for w, g in zip(shape, got)):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(got)}")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} must be on device {device}, got {t.device}")


def _int32(x, name):
    """The library's sizes are int32; ctypes would wrap what is not."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must be an int32, got {x}")
    return x


class Chunk:
    """One batch of chunks in the verify step's layout (device int32 tensors; see sv_chunk)."""

    def __init__(self, seq_offsets, cached, rows: int, max_gamma: int, parents=None):
        B = cached.numel()
        _check(cached, "cached", (torch.int32,), (B,))
        _check(seq_offsets, "seq_offsets", (torch.int32,), (B + 1,), cached.get_device())
        if parents is not None:
            _check(parents, "parents", (torch.int32,), (None,), cached.get_device())
        for t, name in ((seq_offsets, "seq_offsets"), (cached, "cached"), (parents, "parents")):
            if t is not None and not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        self.seq_offsets, self.cached, self.parents = seq_offsets, cached, parents
        self.B, self.rows, self.max_gamma, self.device = B, rows, max_gamma, cached.get_device()
        self.struct = SvChunk(_ptr(seq_offsets), _ptr(cached), _ptr(parents), B, _int32(rows, "rows"),
                              _int32(max_gamma, "max_gamma"), 0)
        self.at = ctypes.addressof(self.struct)


class Rope:
    """Rotary positions: a float32 table [positions, dim], cosines then sines (see sv_rope)."""

    def __init__(self, table, interleaved: bool = False):
        _check(table, "table", (torch.float32,), (None, None))
        if not table.is_contiguous():
            raise ValueError("table must be contiguous")
        self.table, self.device = table, table.get_device()
        self.struct = SvRope(_ptr(table), table.shape[0], table.shape[1], int(interleaved), 0)
        self.at = ctypes.addressof(self.struct)


class PagedCache:
    """A paged key/value cache over the caller's tensors, with the workspace and status word of its calls.

    k, v: [layers, pages, page_size, heads, head_dim], bfloat16, float16 or float8_e4m3fn, of equal strides
    (views of another order, such as head-major pages, are fine; the last dimension is contiguous).
    page_table: int32 [sequences, pages per sequence]; a chunk has as many sequences, or the first of them.
    k_scale, v_scale: float32 [layers, heads] (float8_e4m3fn only).
    Calls of one object share its workspace and must not overlap on the GPU.
    """

    def __init__(self, k, v, page_table, k_scale=None, v_scale=None):
        codes = _CACHES
        _check(k, "k", tuple(codes), (None,) * 5)
        _check(v, "v", (k.dtype,), k.shape, k.get_device())
        if k.stride() != v.stride() or k.stride(4) != 1:
            raise ValueError("k and v must have equal strides and contiguous heads")
        _check(page_table, "page_table", (torch.int32,), (None, None), k.get_device())
        if page_table.shape[0] > 1 and page_table.stride(0) < page_table.shape[1] or page_table.stride(1) != 1:
            raise ValueError("page_table's rows must be contiguous")
        layers, pages, page_size, heads, dim = k.shape
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is not None:
                _check(t, name, (torch.float32,), (layers, heads), k.get_device())
                if not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
        self.k, self.v, self.page_table, self.k_scale, self.v_scale = k, v, page_table, k_scale, v_scale
        self.heads, self.head_dim, self.sequences = heads, dim, page_table.shape[0]
        # of a dimension of extent one the stride says nothing: any valid one does
        st = [k.stride(i) if k.shape[i] > 1 else heads * page_size * dim for i in range(4)]
        width = page_table.stride(0) if page_table.shape[0] > 1 else page_table.shape[1]
        if width != page_table.shape[1]:
            raise ValueError("page_table must be contiguous")
        self.struct = SvCache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(page_table), st[1], st[2], st[3],
                              st[0], codes[k.dtype], layers, pages, page_size, heads, dim, page_table.shape[1], 0)
        self.ws_bytes = spec_cache_workspace_size(self.struct)
        self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=k.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=k.device)
        # addresses that no call changes
        self._at, self._status, self._ws = ctypes.addressof(self.struct), _ptr(self.status), _ptr(self.workspace)
        self._device = k.get_device()

    def _refuse(self, chunk, layer=0, rope=None):
        """What is wrong with a call whose chunk, layer or rotation table is not for this cache. (The calls ask for that
        in line: a function each would cost them half a microsecond.)"""
        if chunk.B > self.sequences:
            raise ValueError(f"page_table has {self.sequences} sequences, the chunk {chunk.B}")
        if chunk.device != self._device:
            raise ValueError(f"chunk must be on {self.k.device}, got device {chunk.device}")
        _int32(layer, "layer")
        raise ValueError(f"rope must be on {self.k.device}, got device {rope.device}")

    def _rows(self, t, name, rows, heads=None):
        """Rows of [heads, head_dim], contiguous within a row: the row stride. These checks and the launch are all
        that a call costs the host, a few microseconds."""
        n, h, d = t.shape if t.dim() == 3 else (0, 0, 0)
        if n < rows or d != self.head_dim or (heads is not None and h != heads):
            raise ValueError(f"{name} must be [{rows}, {heads or 'heads'}, {self.head_dim}], got {tuple(t.shape)}")
        if t.get_device() != self._device:
            raise ValueError(f"{name} must be on {self.k.device}, got {t.device}")
        s0, s1, s2 = t.stride()
        if s2 != 1 or (s1 != d and h > 1):
            raise ValueError(f"{name}'s heads must be contiguous within a row")
        return s0 if n > 1 else h * d

    def _type(self, *ts):
        raise TypeError(f"tensors must share bfloat16 or float16, got {[str(t.dtype) for t in ts]}")

    def _stream(self, stream):
        if stream is not None:
            return stream.cuda_stream
        return torch._C._cuda_getCurrentRawStream(self._device)  # the current stream's handle alone

    def append(self, chunk: Chunk, q, k, v, q_out, rope: Rope | None = None, layer: int = 0, stream=None) -> int:
        """Enqueue spec_cache_append: rotated queries to q_out, rotated keys and values to the cache. q and
        q_out may be None."""
        if chunk.B > self.sequences or chunk.device != self._device or not -2 ** 31 <= layer < 2 ** 31 or (
                rope is not None and rope.device != self._device):
            self._refuse(chunk, layer, rope)
        rows, kind = chunk.rows, k.dtype
        code = _ACTIVATIONS.get(kind)
        if code is None or v.dtype != kind or (q is not None and (q.dtype != kind or q_out.dtype != kind)):
            self._type(*(t for t in (q, k, v, q_out) if t is not None))
        ks = self._rows(k, "k", rows, self.heads)
        if self._rows(v, "v", rows, self.heads) != ks:
            raise ValueError("k and v must have equal row strides")
        qh, qs = 0, 0
        if q is not None:
            qs, qh = self._rows(q, "q", rows), q.shape[1]
            if self._rows(q_out, "q_out", rows, qh) != qh * self.head_dim:
                raise ValueError("q_out must be contiguous")
        return lib.spec_cache_append(self._at, layer, chunk.at, None if rope is None else rope.at, code,
                                     qh, _ptr(q), qs, k.data_ptr(), v.data_ptr(), ks, _ptr(q_out), self._status,
                                     self._stream(stream))

    def attend(self, chunk: Chunk, q, out, lse=None, scale: float | None = None, window: int = 0, layer: int = 0,
               stream=None) -> int:
        """Enqueue spec_cache_attend: attention of the chunk's rotated queries into out (and lse, float32
        [rows, q_heads]). scale: 1 / sqrt(head_dim) by default; window: 0 for none, as any past every length is."""
        if chunk.B > self.sequences or chunk.device != self._device or not -2 ** 31 <= layer < 2 ** 31:
            self._refuse(chunk, layer)
        rows, kind = chunk.rows, q.dtype
        code = _ACTIVATIONS.get(kind)
        if code is None or out.dtype != kind:
            self._type(q, out)
        qs, qh = self._rows(q, "q", rows), q.shape[1]
        if self._rows(out, "out", rows, qh) != qh * self.head_dim:
            raise ValueError("out must be contiguous")
        if lse is not None:
            _check(lse, "lse", (torch.float32,), (None, qh), self._device)
            if lse.shape[0] < rows or not lse.is_contiguous():
                raise ValueError("lse must be contiguous with a row for every chunk row")
        if scale is None:
            scale = self.head_dim ** -0.5
        if not -2 ** 31 <= window < 2 ** 31:
            window = max(-2 ** 31, min(window, 2 ** 31 - 1))
        return lib.spec_cache_attend(self._at, layer, chunk.at, code, qh, q.data_ptr(), qs, scale, window,
                                     out.data_ptr(), _ptr(lse), self._status, self._ws, self.ws_bytes,
                                     self._stream(stream))

    def compact(self, chunk: Chunk, out_num_accepted, out_path, out_cached, stream=None) -> int:
        """Enqueue spec_cache_compact on a verify call's outputs. out_path None: linear drafts. out_cached may
        be the chunk's `cached`."""
        if chunk.B > self.sequences or chunk.device != self._device:
            self._refuse(chunk)
        _check(out_num_accepted, "out_num_accepted", (torch.int32,), (chunk.B,), self._device)
        _check(out_cached, "out_cached", (torch.int32,), (chunk.B,), self._device)
        if out_path is not None:
            _check(out_path, "out_path", (torch.int32,), (None,), self._device)
        if not (out_num_accepted.is_contiguous() and out_cached.is_contiguous() and
                (out_path is None or out_path.is_contiguous())):
            raise ValueError("out_num_accepted, out_path and out_cached must be contiguous")
        return lib.spec_cache_compact(self._at, chunk.at, out_num_accepted.data_ptr(), _ptr(out_path),
                                      out_cached.data_ptr(), self._status, self._stream(stream))

    def status_bits(self) -> int:
        return int(self.status.item()) & 0xFFFFFFFF
