"""Rotary positions, the paged key/value cache and attention over it.

Thin binding like the rest of the package: objects here only hold torch tensors and the C
structures that describe them.

    spec = Rotary([10000.0 ** (-i / 64) for i in range(64)])
    cache = KVCache(k_pages, v_pages)                       # [n_pages, Hkv, page_size, D] bf16
    batch = CacheBatch(q_start, kv_len, table, max_q=1)     # int32, on the device
    q = cache_append(k, v, cache, batch, rotary=spec, q=q)  # k, v [T, Hkv, D], q [T, Hq, D]
    o, lse = fwd_cached(q, cache, batch, Pattern(window=1024, sinks=4))
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import EXPORTED, Pattern, _check, _stream_handle, lib


class _View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class _Rotary(ctypes.Structure):
    _fields_ = [("n_pairs", ctypes.c_int32), ("n_axes", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("freq", ctypes.c_void_p), ("axis", ctypes.c_void_p)]


class _KVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]


class _CacheBatch(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("table_stride", ctypes.c_int64), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("table", ctypes.c_void_p)]


def _declare() -> None:
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    # views, batches, patterns and shapes are made for every call: as packed bytes, whose address is passed
    V = B = S = P = vp
    C, R = ctypes.POINTER(_KVCache), ctypes.POINTER(_Rotary)
    lib.sparse_attn_rotary.argtypes = [V, V, vp, i64, i64, R, S, i32, V, V, vp]
    lib.sparse_attn_cache_append.argtypes = [V, V, C, B, R, vp, i64, i32, V, V, i32, vp]
    lib.sparse_attn_fwd_cached.argtypes = [V, C, B, P, i32, ctypes.c_float, V, vp, vp, sz, vp]
    lib.sparse_attn_fwd_shared.argtypes = [V, C, B, vp, i32, P, i32, ctypes.c_float, V, vp, vp, sz, vp]
    for f in ("sparse_attn_fwd_cached_workspace", "sparse_attn_fwd_shared_workspace"):
        getattr(lib, f).argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
    for f in EXPORTED[EXPORTED.index("sparse_attn_rotary"):]:
        getattr(lib, f).restype = ctypes.c_int


_declare()


# Calls of a few microseconds on the device are common here (one decoding step), so what a call does on
# the host is kept short: attributes are read once, and the device is only switched when it has to be.

_BF16, _I32 = torch.bfloat16, torch.int32
_ref = ctypes.byref


def _rows(where: str, name: str, t, dims: int, device=None):
    """(shape, strides) of a bf16 CUDA tensor of `dims` dimensions with contiguous rows."""
    st = t.stride()
    if t.dtype is not _BF16 or not t.is_cuda or len(st) != dims or st[-1] != 1:
        raise TypeError(f"{where}: {name} must be a {dims}-dimensional bf16 CUDA tensor with contiguous rows")
    if device is not None and t.device != device:
        raise TypeError(f"{where}: {name} is on {t.device}, not on {device}")
    return t.shape, st


def _int32(where: str, name: str, t, dims: int, device) -> None:
    if t.dtype is not _I32 or not t.is_cuda or t.dim() != dims or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise TypeError(f"{where}: {name} must be a {dims}-dimensional int32 CUDA tensor with contiguous rows")
    if t.device != device:
        raise TypeError(f"{where}: {name} is on {t.device}, not on {device}")


def _mismatch(where: str, name: str, shape, want):
    raise ValueError(f"{where}: {name} has the shape {tuple(shape)}, not {tuple(want)}")


# The C structures made for every call, packed (half the time of a ctypes structure).
_pack_view = struct.Struct("@Pqqq").pack      # _View
_pack_shape = struct.Struct("@5i").pack       # _Shape
_pack_pattern = struct.Struct("@7i").pack    # _Pattern
_pack_batch = struct.Struct("@4iqPPP").pack   # _CacheBatch


def _tokens(t, st=None) -> bytes:
    """View of a tensor of tokens [T, H, D]."""
    st = st or t.stride()
    return _pack_view(t.data_ptr(), 0, st[1], st[0])


def _sequences(t, st=None) -> bytes:
    """View of whole sequences [B, H, N, D]."""
    st = st or t.stride()
    return _pack_view(t.data_ptr(), st[0], st[1], st[2])


def _empty(shape, dtype, device, stream):
    """Memory for a call on ``stream``: taken there, so that what used it before is done by then, and so
    that a workspace is not handed out again before the kernels are done with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _call(fn, where: str, device, stream, *args) -> None:
    """Call fn(*args, stream handle) with `device` current."""
    index = device.index
    if torch.cuda.current_device() == index:
        status = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream_handle(stream, device))
    if status:
        _check(status, "sparse_attn_" + where)


def _raw_stream(index: int) -> int:
    """Handle of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(index)


if not hasattr(torch._C, "_cuda_getCurrentRawStream"):  # a torch without CUDA, or without the short way
    def _raw_stream(index: int) -> int:  # noqa: F811
        return torch.cuda.current_stream(index).cuda_stream


class Rotary:
    """Which pairs of a row turn, how fast (radians a position) and along which axis of the
    position.  ``freq`` holds one number per pair; ``axis`` one index per pair (default 0).
    Pairs are elements (j, j + len(freq)) or, ``interleaved``, (2j, 2j + 1); elements behind the
    last pair stay."""

    def __init__(self, freq, axis=None, interleaved: bool = False, n_axes: int | None = None):
        freq = [float(f) for f in freq]
        if axis is not None:
            axis = [int(a) for a in axis]
            if len(axis) != len(freq):
                raise ValueError("one axis per frequency")
        self.n_axes = n_axes if n_axes is not None else (max(axis) + 1 if axis else 1)
        self.n_pairs, self.interleaved = len(freq), bool(interleaved)
        self._freq = (ctypes.c_double * max(len(freq), 1))(*freq)
        self._axis = (ctypes.c_int32 * max(len(axis), 1))(*axis) if axis is not None else None
        self._struct = _Rotary(len(freq), self.n_axes, int(self.interleaved), ctypes.addressof(self._freq),
                               ctypes.addressof(self._axis) if axis is not None else None)
        self._ref = _ref(self._struct)


class KVCache:
    """Keys and values in pages: two bf16 CUDA tensors [n_pages, Hkv, page_size, D] of equal
    strides (any order of heads and places in memory; rows of D contiguous)."""

    def __init__(self, k_pages, v_pages):
        _rows("KVCache", "k_pages", k_pages, 4)
        _rows("KVCache", "v_pages", v_pages, 4, k_pages.device)
        if k_pages.shape != v_pages.shape or k_pages.stride() != v_pages.stride():
            raise ValueError("KVCache: k_pages and v_pages differ in shape or strides")
        self.k, self.v, self.device = k_pages, v_pages, k_pages.device
        n, self.Hkv, self.page_size, self.D = k_pages.shape
        st = k_pages.stride()
        self._struct = _KVCache(k_pages.data_ptr(), v_pages.data_ptr(), n, self.page_size, self.Hkv, self.D, st[0],
                                st[1], st[2])
        self._ref = _ref(self._struct)


class CacheBatch:
    """A batch over a cache: ``q_start`` [B + 1] rows of the token tensors where each sequence's
    new tokens begin (ascending from 0), ``kv_len`` [B] cached tokens (new ones included),
    ``table`` [B, max_pages] pages.  int32 CUDA tensors; their contents are read when a kernel
    runs, so a captured graph follows them.  Tokens whose place lies behind the table are not in the
    cache.  ``max_q``: most new tokens of one sequence, as far as known.  Results do not depend on
    it, the choice of kernels does: left out, the average is taken, and a long piece among many
    single tokens then runs on the kernel for few rows (255 single tokens and a piece of 512, 32/8
    heads of 128: 224 us with ``max_q=512``, 442 without).  Give it where pieces and single tokens
    mix."""

    def __init__(self, q_start, kv_len, table, max_q: int | None = None):
        dev = q_start.device
        _int32("CacheBatch", "q_start", q_start, 1, dev)
        _int32("CacheBatch", "kv_len", kv_len, 1, dev)
        _int32("CacheBatch", "table", table, 2, dev)
        B = kv_len.shape[0]
        if q_start.shape[0] != B + 1 or table.shape[0] != B:
            raise ValueError("CacheBatch: q_start [B + 1], kv_len [B] and table [B, max_pages] disagree on B")
        self.q_start, self.kv_len, self.table, self.max_q, self.device = q_start, kv_len, table, max_q, dev
        self._B = B
        self._rest = (max_q or 0, table.shape[1], table.stride(0) if B > 1 else table.shape[1], q_start.data_ptr(),
                      kv_len.data_ptr(), table.data_ptr())

    def _c(self, T: int) -> bytes:
        return _pack_batch(self._B, T, *self._rest)


def _rotate(where, q, k, positions, spec, backward, q_out, k_out, stream):
    shape, st = _rows(where, "q", q, 4)
    B, Hq, N, D = shape
    dev = q.device
    _int32(where, "positions", positions, 3, dev)
    n_axes, Bp, Np = positions.shape
    if n_axes != spec.n_axes or (Bp != B and Bp != 1) or Np != N:
        raise ValueError(f"{where}: positions must be [{spec.n_axes}, {B} or 1, {N}]")
    qv = _sequences(q, st)
    if q_out is None:
        q_out = _empty(shape, _BF16, dev, stream)
        ov = _sequences(q_out)
    else:
        oshape, ost = _rows(where, "q_out", q_out, 4, dev)
        if oshape != shape:
            _mismatch(where, "q_out", oshape, shape)
        ov = _sequences(q_out, ost)
    kv = okv = None
    Hkv = 0
    if k is not None:
        kshape, kst = _rows(where, "k", k, 4, dev)
        Hkv = kshape[1]
        if kshape[0] != B or kshape[2] != N or kshape[3] != D:
            _mismatch(where, "k", kshape, (B, Hkv, N, D))
        if k_out is None:
            k_out = _empty(kshape, _BF16, dev, stream)
            okv = _sequences(k_out)
        else:
            oshape, ost = _rows(where, "k_out", k_out, 4, dev)
            if oshape != kshape:
                _mismatch(where, "k_out", oshape, kshape)
            okv = _sequences(k_out, ost)
        kv = _sequences(k, kst)
    elif k_out is not None:
        raise ValueError(f"{where}: k_out without k")
    pst = positions.stride()
    _call(lib.sparse_attn_rotary, "rotary", dev, stream, qv, kv, positions.data_ptr(), pst[0],
          pst[1] if Bp > 1 else 0, spec._ref, _pack_shape(B, Hq, Hkv, N, D), backward, ov, okv)
    return q_out, k_out


def rotary(q, k, positions, spec: Rotary, q_out=None, k_out=None, stream=None):
    """(q', k') rotated by their positions.  q [B, Hq, N, D], k [B, Hkv, N, D] (or None), bf16 CUDA
    tensors with contiguous rows, any other strides; positions int32 [n_axes, B, N] or
    [n_axes, 1, N].  An output may be its input.  Asynchronous on ``stream``."""
    return _rotate("rotary", q, k, positions, spec, 0, q_out, k_out, stream)


def rotary_bwd(dq, dk, positions, spec: Rotary, q_out=None, k_out=None, stream=None):
    """Gradients of ``rotary``'s inputs from those of its outputs (the rotation by the negated
    angles).  Arguments as ``rotary``."""
    return _rotate("rotary_bwd", dq, dk, positions, spec, 1, q_out, k_out, stream)


def cache_append(k, v, cache: KVCache, batch: CacheBatch, rotary: Rotary | None = None, positions=None,
                 pos_offset: int = 0, q=None, q_out=None, stream=None):
    """Write the new tokens' keys and values [T, Hkv, D] to their places in the cache, keys rotated
    by ``rotary`` on the way.  With ``q`` [T, Hq, D] the queries are rotated in the same launch and
    returned (in ``q_out`` if given, which may be ``q``).  ``positions`` int32 [n_axes, T] replaces
    the tokens' positions in the cache (+ ``pos_offset``).  Asynchronous on ``stream``."""
    where = "cache_append"
    dev = cache.device
    shape, kst = _rows(where, "k", k, 3, dev)
    T = shape[0]
    if shape[1] != cache.Hkv or shape[2] != cache.D:
        _mismatch(where, "k", shape, (T, cache.Hkv, cache.D))
    vshape, vst = _rows(where, "v", v, 3, dev)
    if vshape != shape:
        _mismatch(where, "v", vshape, shape)
    if batch.device != dev:
        raise TypeError(f"{where}: batch is on {batch.device}, not on {dev}")
    pos_ptr, pos_stride = None, 0
    if positions is not None:
        if rotary is None:
            raise ValueError(f"{where}: positions without rotary")
        _int32(where, "positions", positions, 2, dev)
        if tuple(positions.shape) != (rotary.n_axes, T):
            _mismatch(where, "positions", positions.shape, (rotary.n_axes, T))
        pos_ptr, pos_stride = positions.data_ptr(), positions.stride(0)
    qv = ov = None
    Hq = 0
    if q is not None:
        if rotary is None:
            raise ValueError(f"{where}: q without rotary")
        qshape, qst = _rows(where, "q", q, 3, dev)
        Hq = qshape[1]
        if qshape[0] != T or qshape[2] != cache.D:
            _mismatch(where, "q", qshape, (T, Hq, cache.D))
        if q_out is None:
            q_out = _empty(qshape, _BF16, dev, stream)
            ov = _tokens(q_out)
        else:
            oshape, ost = _rows(where, "q_out", q_out, 3, dev)
            if oshape != qshape:
                _mismatch(where, "q_out", oshape, qshape)
            ov = _tokens(q_out, ost)
        qv = _tokens(q, qst)
    elif q_out is not None:
        raise ValueError(f"{where}: q_out without q")
    _call(lib.sparse_attn_cache_append, "cache_append", dev, stream, _tokens(k, kst),
          _tokens(v, vst), cache._ref, batch._c(T), rotary._ref if rotary is not None else None, pos_ptr,
          pos_stride, int(pos_offset), qv, ov, Hq)
    return q_out


def _workspace(where: str, T: int, Hq: int, Hkv: int, D: int) -> int:
    n = ctypes.c_size_t(0)
    fn = f"sparse_attn_{where}_workspace"
    _check(getattr(lib, fn)(T, Hq, Hkv, D, ctypes.byref(n)), fn)
    return n.value


def fwd_cached_workspace_bytes(T: int, Hq: int, Hkv: int, D: int) -> int:
    return _workspace("fwd_cached", T, Hq, Hkv, D)


def fwd_shared_workspace_bytes(T: int, Hq: int, Hkv: int, D: int) -> int:
    return _workspace("fwd_shared", T, Hq, Hkv, D)


def _attend(fn, where, q, cache, batch, prefix, pattern, scale, out, lse, workspace, stream):
    dev, p = cache.device, pattern
    shape, st = _rows(where, "q", q, 3, dev)
    T, Hq, D = shape
    if D != cache.D:
        _mismatch(where, "q", shape, (T, Hq, cache.D))
    if batch.device != dev:
        raise TypeError(f"{where}: batch is on {batch.device}, not on {dev}")
    if out is None:
        out = _empty(shape, _BF16, dev, stream)
        ov = _tokens(out)
    else:
        oshape, ost = _rows(where, "out", out, 3, dev)
        if oshape != shape:
            _mismatch(where, "out", oshape, shape)
        ov = _tokens(out, ost)
    if lse is None:
        lse = _empty((T, Hq), torch.float32, dev, stream)
    elif lse.dtype is not torch.float32 or lse.device != dev or not lse.is_contiguous() or lse.shape != (T, Hq):
        raise TypeError(f"{where}: lse must be a contiguous fp32 tensor [T, Hq] on {dev}")
    if workspace is None:
        workspace = _empty(max(_workspace(where, T, Hq, cache.Hkv, D), 1), torch.uint8, dev, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise TypeError(f"{where}: workspace must be a contiguous tensor on {dev}")
    _call(fn, where, dev, stream, _tokens(q, st), cache._ref, batch._c(T), *prefix,
          _pack_pattern(p.causal, p.window, p.sinks, p.stride, p.n_global, p.area, p.summary), Hq,
          scale if scale is not None else 1.0 / math.sqrt(D), ov, lse.data_ptr(), workspace.data_ptr(),
          workspace.nbytes)
    return out, lse


def fwd_cached(q, cache: KVCache, batch: CacheBatch, pattern: Pattern, scale: float | None = None, out=None, lse=None,
               workspace=None, stream=None):
    """Attention of new tokens q [T, Hq, D] over the cache: O [T, Hq, D] bf16 and LSE [T, Hq] fp32.

    ``pattern`` is causal with window, sinks and n_global.  Rows of no sequence keep what ``out``
    and ``lse`` held; rows that see nothing get 0 and -inf, rows that see a score of NaN or +inf get
    NaN for both.  ``workspace``: at least ``fwd_cached_workspace_bytes`` bytes, not shared by
    calls that may run at the same time.  Asynchronous on ``stream``."""
    return _attend(lib.sparse_attn_fwd_cached, "fwd_cached", q, cache, batch, (), pattern, scale, out, lse, workspace,
                   stream)


def fwd_shared(q, cache: KVCache, batch: CacheBatch, prefix_table, prefix_len: int, pattern: Pattern,
               scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """``fwd_cached`` for sequences that all begin with one prefix of ``prefix_len`` tokens in the
    pages ``prefix_table`` (int32 CUDA tensor), read once for all of them.  ``batch`` describes what
    follows the prefix.  ``workspace``: at least ``fwd_shared_workspace_bytes`` bytes."""
    prefix_len = int(prefix_len)
    if prefix_table is None:
        if prefix_len:
            raise ValueError("fwd_shared: prefix_len without prefix_table")
        ptr = None
    else:
        _int32("fwd_shared", "prefix_table", prefix_table, 1, cache.device)
        if prefix_len > prefix_table.shape[0] * cache.page_size:
            raise ValueError("fwd_shared: prefix_table holds fewer than prefix_len tokens")
        ptr = prefix_table.data_ptr()
    return _attend(lib.sparse_attn_fwd_shared, "fwd_shared", q, cache, batch, (ptr, prefix_len), pattern, scale, out,
                   lse, workspace, stream)
