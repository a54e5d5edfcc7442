"""ctypes binding of the C ABI in ``include/kv_cache.h`` (argument marshalling only).

What a decode instance does with the KV it was handed: :class:`KVCache` appends new tokens to
one shard pool and attends to it, :func:`rotary_table` fills the table of rotations. Every step
runs in the CUDA library; there is no fallback.
"""
from __future__ import annotations

import ctypes
import struct

import numpy as np

from .kv_relayout import (KVRelayoutError, KvrLayout, _contiguous, _Layout, _nbytes, _ptr,
                          _stream_handle, library)

DTYPE_F16 = 3
INTERLEAVED = 1
ROTATE_LAST = 2
FLAGS = {1: "request index", 2: "position", 4: "length", 8: "block id", 16: "wait"}
SCALINGS = {"linear": 1, "base": 2, "ramp": 3, "bands": 4}
CACHE_EXPORTS = ("kv_cache_create", "kv_cache_destroy", "kv_cache_workspace_bytes",
                 "kv_cache_append", "kv_cache_attend", "kv_cache_status",
                 "kv_cache_rotary_table")

# kvc_append and kvc_attend as the C header lays them out (no padding between their fields)
_APPEND = struct.Struct("=iiQQQqiiQQqqqqQiiIiiiQQqqqq")
_ATTEND = struct.Struct("=iiiifiQQqiiQQQqqqqqq")


class KvcDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("num_layers", "num_components", "kv_heads", "head_dim", "value_dim", "dtype",
                 "block_size", "per_head")] + \
               [("num_blocks", ctypes.c_int64), ("pool", ctypes.c_void_p),
                ("layout", ctypes.POINTER(KvrLayout)), ("scales", ctypes.c_void_p),
                ("query_heads", ctypes.c_int32), ("max_requests", ctypes.c_int32),
                ("max_new", ctypes.c_int32)]


class KvcScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("original", ctypes.c_int32),
                ("factor", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("magnitude", ctypes.c_double)]


_bound = None


def _library() -> ctypes.CDLL:
    global _bound
    if _bound is None:
        lib = library()
        i32, p = ctypes.c_int32, ctypes.c_void_p
        for name, args in (("kv_cache_create", [p, p]),
                           ("kv_cache_workspace_bytes", [p, i32, p]),
                           ("kv_cache_append", [p, i32, p, p]),
                           ("kv_cache_attend", [p, i32, p, p]), ("kv_cache_status", [p, p]),
                           ("kv_cache_rotary_table", [p, i32, i32, ctypes.c_double, p])):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = i32, args
        lib.kv_cache_destroy.restype, lib.kv_cache_destroy.argtypes = None, [p]
        _bound = lib
    return _bound


def rotary_table(rows, rotary_dim, base=10000.0, scaling=None):
    """Cosines and sines of positions [0, rows): a float32 numpy array [rows][rotary_dim] to
    copy to the device (``kv_cache_rotary_table``). ``scaling``: None or dict(kind="linear" |
    "base" | "ramp" | "bands", factor=..., original=..., beta_fast=32.0, beta_slow=1.0,
    magnitude=0.0)."""
    out = np.empty((rows, rotary_dim), dtype=np.float32)
    sc = None
    if scaling is not None:
        s = dict(scaling)
        kind = s.pop("kind")
        if kind not in SCALINGS:
            raise ValueError(f"scaling kind {kind!r} is none of {sorted(SCALINGS)}")
        sc = KvcScaling(SCALINGS[kind], int(s.pop("original", 0)), float(s.pop("factor")),
                        float(s.pop("beta_fast", 32.0)), float(s.pop("beta_slow", 1.0)),
                        float(s.pop("magnitude", 0.0)))
        if s:
            raise ValueError(f"unknown scaling entries {sorted(s)}")
    st = _library().kv_cache_rotary_table(out.ctypes.data, int(rows), int(rotary_dim),
                                          float(base), ctypes.byref(sc) if sc else None)
    if st != 0:
        raise KVRelayoutError(st, "kv_cache_rotary_table")
    return out


def _desc(pool, layout, scales, per_head, geometry):
    """The C descriptor and the host objects that it points to."""
    d = KvcDesc()
    lay = None if layout is None else _Layout(**layout)
    sc = None if scales is None else np.ascontiguousarray(scales, dtype=np.float32)
    for name in ("num_layers", "num_components", "kv_heads", "head_dim", "dtype", "num_blocks",
                 "query_heads", "max_requests", "max_new", "value_dim"):
        setattr(d, name, int(geometry[name]))
    d.block_size, d.per_head = int(geometry["block"]), int(bool(per_head)) if sc is not None else 0
    d.pool = None if pool is None else _ptr(pool)
    d.layout = ctypes.pointer(lay.layout) if lay is not None else None
    d.scales = sc.ctypes.data if sc is not None else None
    return d, (lay, sc)


def workspace_bytes(sm_count, pool=1 << 40, layout=None, scales=None, per_head=False, **geometry):
    """Validate a cache's geometry on the host; the device bytes of its workspace."""
    d, keep = _desc(pool, layout, scales, per_head, _defaults(geometry))
    out = ctypes.c_int64()
    st = _library().kv_cache_workspace_bytes(ctypes.byref(d), int(sm_count), ctypes.byref(out))
    if st != 0:
        raise KVRelayoutError(st, "kv_cache_workspace_bytes")
    return out.value


def _defaults(g):
    return dict(dict(query_heads=0, max_requests=1, max_new=1, value_dim=0), **g)


class KVCache:
    """One shard pool of a decode side: append tokens to it, attend to it.

    ``pool``: a contiguous tensor (or address) [num_layers][num_components][num_blocks][block]
    [kv_heads][head_dim] -- the decode pool that a :class:`RelayoutPlan` wrote -- with ``kv_heads``
    the shard's heads; or ``layout=layout_of_views([views])`` for any strided one. ``dtype``:
    DTYPE_BF16, DTYPE_F16 or DTYPE_FP8_E4M3, the last with ``scales`` [L][C] (``per_head``:
    [L][C][H]) as the relayout's conversion takes them. Two components hold keys and values
    (head_dim a multiple of 16, at most 256), one a latent (head_dim 576, of which the first
    512 are the values). ``query_heads`` (0: append only), ``max_requests`` and ``max_new`` size
    the workspace of the attention calls (:func:`workspace_bytes`: 40 MB for latents, 5 to 10 MB for
    keys and values, whatever the pool's size); calls on different streams that share a cache must
    be ordered, host threads need not be. Tensors that the calls do not hold for are ValueErrors, what the C library
    refuses is a KVRelayoutError.

    Calls run on torch's current stream, or on ``stream`` (a torch stream or a handle). Results that a
    call makes belong to that stream, as those of torch's own operations do: used on another one,
    they need its order and ``record_stream``; and so do inputs of another stream. There is no
    backward pass: where gradients are recorded, tensors that require one are refused.
    """

    def __init__(self, pool, *, num_layers, num_components, kv_heads, head_dim, block,
                 num_blocks, dtype, scales=None, per_head=False, layout=None, query_heads=0,
                 max_requests=1, max_new=1, value_dim=0):
        self._h = None
        g = dict(num_layers=num_layers, num_components=num_components, kv_heads=kv_heads,
                 head_dim=head_dim, block=block, num_blocks=num_blocks, dtype=dtype,
                 query_heads=query_heads, max_requests=max_requests, max_new=max_new,
                 value_dim=value_dim)
        es = 1 if dtype == 2 else 2
        if layout is not None:
            shape, elem = layout.get("shape"), layout.get("elem_bytes")
            need = (num_blocks, block, kv_heads, head_dim)
            if elem is not None and elem != es:
                raise ValueError(f"views hold {elem}-byte elements; the cache holds {es}-byte ones")
            if shape is not None and any(h < n for h, n in zip(shape, need)):
                raise ValueError(f"views are {list(shape)} ([block][token][head][dim]); "
                                 f"the geometry addresses {list(need)}")
            if len(layout["bases"]) != num_layers * num_components:
                raise ValueError(f"{len(layout['bases'])} views; the geometry has "
                                 f"{num_layers} layers of {num_components} components")
        elif pool is not None:
            if not _contiguous(pool):
                raise ValueError("pool is not contiguous: describe it with a layout")
            need = num_layers * num_components * num_blocks * block * kv_heads * head_dim * es
            have = _nbytes(pool)
            if have is not None and have < need:
                raise ValueError(f"pool holds {have} bytes; the geometry addresses {need}")
        if scales is not None:
            n = num_layers * num_components * (kv_heads if per_head else 1)
            if np.size(scales) != n:
                raise ValueError(f"{np.size(scales)} scales; {n} expected")
        d, _ = _desc(pool, layout, scales, per_head, g)
        h = ctypes.c_void_p()
        st = _library().kv_cache_create(ctypes.byref(d), ctypes.byref(h))
        if st != 0:
            raise KVRelayoutError(st, "kv_cache_create")
        import torch
        lib = _library()
        self._h, self._pool, self._torch = h.value, (pool, layout), torch
        self._append, self._attend = lib.kv_cache_append, lib.kv_cache_attend
        self._index = torch.cuda.current_device()
        self._device = torch.device("cuda", self._index)
        self._i32, self._f32 = torch.int32, torch.float32
        self._types = {torch.bfloat16: 1, torch.float16: DTYPE_F16}
        self._raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        self.kv_heads, self.head_dim, self.query_heads = kv_heads, head_dim, query_heads
        self.value_dim = value_dim or (512 if num_components == 1 else head_dim)
        self.latent = num_components == 1
        self._default_scale = head_dim ** -0.5
        self._row_bytes = (2 * kv_heads * head_dim, 2 * head_dim)

    # -- arguments ---------------------------------------------------------------
    #
    # A decode step calls these for every layer, and they cost about as much as the small kernels
    # behind them: contiguous tensors are looked at where they are used, in as few Python operations
    # as that takes, and only others (and wrong ones) reach the methods below.

    def _handle(self):
        if self._h is None:
            raise RuntimeError("cache already closed")
        return self._h

    def _refuse_gradients(self):
        """For tensors of which one requires a gradient: the results would silently have none."""
        if self._torch.is_grad_enabled():
            raise ValueError("a tensor here requires a gradient, and these calls have none: "
                             "call them under torch.no_grad() or detach it")

    def _new(self, shape, dtype, stream):
        """A result's memory, from the allocator's share of the stream that the kernel writes it on: memory
        of torch's current stream may still be in use by what is queued there."""
        if stream is None:
            return self._torch.empty(shape, dtype=dtype, device=self._device)
        cuda, handle = self._torch.cuda, _stream_handle(stream) or 0
        on = cuda.ExternalStream(handle, device=self._device) if handle > 1 else \
            cuda.default_stream(self._device)              # (0 and 1: the legacy default stream)
        with cuda.stream(on):
            return self._torch.empty(shape, dtype=dtype, device=self._device)

    def _rows(self, t, name, shape, dtype=None):
        """Byte strides of a tensor of head rows but the last dimension's, once it is checked."""
        if t.shape == shape and t.get_device() == self._index and \
                (t.dtype is dtype if dtype is not None else t.dtype in self._types):
            if t.is_contiguous():
                row = 2 * shape[-1]
                if len(shape) == 3:
                    return shape[1] * row, row
                return shape[1] * shape[2] * row, shape[2] * row, row
            st = t.stride()
            if st[-1] == 1:
                return tuple(2 * x if e > 1 else 0 for x, e in zip(st[:-1], shape[:-1]))
        raise ValueError(f"{name} is {t.dtype} {list(t.shape)} on {t.device} with strides "
                         f"{list(t.stride())}; expected {dtype or 'bfloat16 or float16'} "
                         f"{list(shape)} on {self._device}, rows contiguous")

    def _list(self, t, name, n):
        if t.dtype is self._i32 and t.shape == (n,) and t.is_contiguous() and \
                t.get_device() == self._index:
            return t.data_ptr()
        raise ValueError(f"{name} is {t.dtype} {list(t.shape)} on {t.device}; expected "
                         f"contiguous int32 [{n}] on {self._device}")

    def _table(self, t):
        if t.dtype is self._i32 and t.dim() == 2 and t.get_device() == self._index:
            rows, width = t.shape
            if t.is_contiguous():
                return t.data_ptr(), width, rows, width
            stride, one = t.stride()
            if one == 1 or width <= 1:
                return t.data_ptr(), stride, rows, width     # (rows may overlap: they are only read)
        raise ValueError(f"block table is {t.dtype} {list(t.shape)} on {t.device}; expected "
                         f"int32 [rows][width] on {self._device}, rows contiguous")

    # -- calls -------------------------------------------------------------------

    def append(self, layer, k, v, requests, positions, block_table, *, rotary=None,
               interleaved=False, rotate_last=False, q=None, q_out=None, stream=None):
        """Append tokens to ``layer``: ``k`` and ``v`` [T][H][D] (``v`` None for latents), token t
        of request ``requests[t]`` (a row of ``block_table``) at ``positions[t]``, negative for
        padding. ``rotary``: the table of :func:`rotary_table` on the device, by which the first
        (``rotate_last``: the last) of each row's elements are rotated; ``q`` [T][heads][dim], where
        given, is rotated into ``q_out`` (a new tensor by default). Returns ``q_out``."""
        if (v is None) != self.latent:
            raise ValueError("a latent cache has no values, others need them")
        if k.requires_grad or (v is not None and v.requires_grad) or (q is not None and q.requires_grad):
            self._refuse_gradients()
        index, i32, dtype = self._index, self._i32, k.dtype
        T = k.shape[0]
        shape, line = (T, self.kv_heads, self.head_dim), (T,)
        code = self._types.get(dtype)
        ks = self._row_bytes if code is not None and k.shape == shape and k.is_contiguous() and \
            k.get_device() == index else self._rows(k, "k", shape)
        if v is None:
            vp, vs = 0, (0, 0)
        else:
            vp, vs = v.data_ptr(), self._row_bytes
            if not (v.dtype is dtype and v.shape == shape and v.is_contiguous() and
                    v.get_device() == index):
                vs = self._rows(v, "v", shape, dtype)
        ids, stride, rows, width = self._table(block_table)
        rot = rot_rows = rot_dim = q_heads = q_dim = qp = qo = 0
        qs = os = (0, 0)
        if rotary is not None:
            if rotary.dtype is not self._f32 or rotary.dim() != 2 or \
                    not rotary.is_contiguous() or rotary.get_device() != index:
                raise ValueError("the rotation table is contiguous float32 [positions][rotated] "
                                 f"on {self._device}")
            rot, (rot_rows, rot_dim) = rotary.data_ptr(), rotary.shape
        if q is not None:
            shape = q.shape
            if len(shape) != 3 or shape[0] != T:
                raise ValueError(f"q is {list(shape)}; expected [{T}][heads][dim]")
            _, q_heads, q_dim = shape
            plain = (2 * q_heads * q_dim, 2 * q_dim)
            qs = plain if q.dtype is dtype and q.is_contiguous() and q.get_device() == index else \
                self._rows(q, "q", shape, dtype)
            if q_out is None:
                q_out = self._new(shape, dtype, stream)
            os = plain if q_out.dtype is dtype and q_out.shape == shape and q_out.is_contiguous() and \
                q_out.get_device() == index else self._rows(q_out, "q_out", shape, dtype)
            qp, qo = q.data_ptr(), q_out.data_ptr()
        for t, name in ((requests, "requests"), (positions, "positions")):
            if not (t.dtype is i32 and t.shape == line and t.is_contiguous() and t.get_device() == index):
                self._list(t, name, T)
        st = self._append(
            self._handle(), layer,
            _APPEND.pack(T, code, requests.data_ptr(), positions.data_ptr(), ids, stride, rows, width,
                         k.data_ptr(), vp, *ks, *vs, rot, rot_rows, rot_dim,
                         (INTERLEAVED if interleaved else 0) | (ROTATE_LAST if rotate_last else 0),
                         q_heads, q_dim, 0, qp, qo, *qs, *os),
            self._raw_stream(index) if stream is None else _stream_handle(stream))
        if st != 0:
            raise KVRelayoutError(st, "kv_cache_append")
        return q_out

    def attend(self, layer, q, lengths, block_table, *, out=None, lse=None, scale=None, window=0,
               stream=None):
        """Attention of each request's newest tokens over ``layer``: ``q`` [R][new][Hq][D], or
        [R][Hq][D] for one; ``lengths`` int32 [R] counts the cached tokens, the newest included.
        ``scale``: D ** -0.5 by default; ``window`` > 0: only that many keys, the token's own
        included. Returns (out, lse): ``out`` like q with ``value_dim`` elements, ``lse`` float32
        [R][new][Hq], new tensors by default (``lse=False``: none)."""
        if q.requires_grad:
            self._refuse_gradients()
        index, dtype, shape, heads = self._index, q.dtype, q.shape, self.query_heads
        n = len(shape)
        if n == 4:
            R, m = shape[0], shape[1]
            rows = (R, m, heads)
        elif n == 3:
            R, m = shape[0], 1
            rows = (R, heads)
        else:
            raise ValueError(f"q is {list(shape)}; expected [R][new][heads][dim]")
        q_row, out_row = 2 * self.head_dim, 2 * self.value_dim
        code = self._types.get(dtype)
        if code is not None and shape == rows + (self.head_dim,) and q.is_contiguous() and \
                q.get_device() == index:
            qs = m * heads * q_row, heads * q_row, q_row
        else:
            qs = self._rows(q, "q", rows + (self.head_dim,))
            qs = qs if n == 4 else (qs[0], 0, qs[1])
        line = rows + (self.value_dim,)
        if out is None:
            out = self._new(line, dtype, stream)
        if out.dtype is dtype and out.shape == line and out.is_contiguous() and out.get_device() == index:
            os = m * heads * out_row, heads * out_row, out_row
        else:
            os = self._rows(out, "out", line, dtype)
            os = os if n == 4 else (os[0], 0, os[1])
        if lse is None:
            lse = self._new(rows, self._f32, stream)
        if lse is False:
            lse, lp = None, 0
        elif lse.dtype is self._f32 and lse.shape == rows and lse.is_contiguous() and \
                lse.get_device() == index:
            lp = lse.data_ptr()
        else:
            raise ValueError(f"lse is {lse.dtype} {list(lse.shape)}; expected contiguous "
                             f"float32 {list(rows)} on {self._device}")
        if not (lengths.dtype is self._i32 and lengths.shape == (R,) and lengths.is_contiguous() and
                lengths.get_device() == index):
            self._list(lengths, "lengths", R)
        st = self._attend(
            self._handle(), layer,
            _ATTEND.pack(R, m, code, window, self._default_scale if scale is None else scale, 0,
                         lengths.data_ptr(), *self._table(block_table),
                         q.data_ptr(), out.data_ptr(), lp, *qs, *os),
            self._raw_stream(index) if stream is None else _stream_handle(stream))
        if st != 0:
            raise KVRelayoutError(st, "kv_cache_attend")
        return out, lse

    def check(self):
        """Wait for the device; raise KVRelayoutError (KVR_ERR_DEVICE_BOUNDS) if a call since
        the last check met a request index, position, length or block id out of range (what
        was out of range was neither read nor written)."""
        flags = ctypes.c_uint32()
        st = _library().kv_cache_status(self._handle(), ctypes.byref(flags))
        if st != 0:
            what = ", ".join(n for b, n in FLAGS.items() if flags.value & b)
            raise KVRelayoutError(st, f"kv_cache_status: {what} out of range" if what
                                  else "kv_cache_status")

    def close(self):
        if getattr(self, "_h", None) is not None:
            _library().kv_cache_destroy(self._h)
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
