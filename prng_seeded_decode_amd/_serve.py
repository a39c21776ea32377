"""ctypes binding of the serving operators (seedlm_serve.h): argument marshalling only.

Each operator has a function for a single call and a call object whose arguments are
checked and marshalled once, for loops that repeat a call on the same buffers (a serving
step, a captured graph): calling the object only crosses the C ABI.  A call object keeps
its tensors alive; their contents may change between calls, their storage may not.
"""
from __future__ import annotations

import ctypes

from ._binding import OK, SeedLMError, _dtype_code, _stream_ptr, lib

MAX_REQUESTS = 4096
MAX_RANK = 256

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
_INT32_MAX = 2 ** 31 - 1  # a ctypes field would take a larger number modulo 2^32


class _PlanArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("lens", "fresh", "table", "ring", "ring_state", "lens_out",
                                   "ring_state_out", "offsets", "rows", "positions", "slots",
                                   "ok", "spans")] + [
        ("table_stride", _i64), ("requests", _i32), ("page_size", _i32), ("max_pages", _i32),
        ("pool", _i32), ("tokens", _i32)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("pages", _i64), ("page_stride", _i64),
                ("token_stride", _i64), ("head_stride", _i64), ("page_size", _i32),
                ("kv_heads", _i32), ("head_dim", _i32)]


class _AppendArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("q", "k", "v", "q_out", "cos", "sin", "positions",
                                   "slots")] + [
        ("cache", _Cache), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
        ("q_out_stride", _i64), ("tokens", _i32), ("heads", _i32), ("rot", _i32),
        ("table_len", _i32), ("interleaved", _i32), ("x_dtype", _i32)]


class _AttendArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("q", "out", "table", "rows", "lens")] + [
        ("cache", _Cache), ("q_stride", _i64), ("out_stride", _i64), ("table_stride", _i64),
        ("queries", _i32), ("table_rows", _i32), ("heads", _i32), ("max_pages", _i32), ("max_len", _i32),
        ("x_dtype", _i32), ("scale", ctypes.c_float)]


class _QCache(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("k", "v", "k_scale", "v_scale")] + [
        (n, _i64) for n in ("pages", "page_stride", "token_stride", "head_stride",
                            "scale_page_stride", "scale_token_stride", "scale_head_stride")] + [
        (n, _i32) for n in ("page_size", "kv_heads", "head_dim", "bits", "group")]


class _QAppendArgs(ctypes.Structure):
    _fields_ = [("cache", _QCache) if f[0] == "cache" else f for f in _AppendArgs._fields_]


class _QReadArgs(ctypes.Structure):
    _fields_ = [("k_out", _vp), ("v_out", _vp), ("slots", _vp), ("cache", _QCache),
                ("k_stride", _i64), ("v_stride", _i64), ("tokens", _i32), ("y_dtype", _i32)]


class _QAttendArgs(ctypes.Structure):
    _fields_ = [("cache", _QCache) if f[0] == "cache" else f for f in _AttendArgs._fields_]


class _LoraSite(ctypes.Structure):
    _fields_ = [("x", _vp), ("A", _vp), ("B", _vp), ("base", _vp), ("y", _vp), ("rows", _i64),
                ("cols", _i64), ("rank", _i32)]


def _on_device(tensors):
    """The one device of the tensors, which has to be the current one."""
    import torch

    device = tensors[0].device
    if any(t.device != device or not t.is_cuda for t in tensors):
        raise ValueError("all tensors must be on one device")
    if device.index != torch.cuda.current_device():
        raise ValueError("the tensors' device must be the current one")
    return device.index


def _ints(what, t, n):
    import torch

    if t.dtype != torch.int32 or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{what} must be a contiguous int32 tensor of {n} elements")
    return t.data_ptr()


def _table(table):
    import torch

    if table.dtype != torch.int32 or table.dim() != 2:
        raise ValueError("table must be an int32 tensor [rows][max_pages]")
    if table.shape[1] > 1 and table.stride(1) != 1:
        raise ValueError("the rows of table must be contiguous")
    return (table.data_ptr(), table.shape[1],
            table.stride(0) if table.shape[0] > 1 else table.shape[1])


def _heads(what, t, tokens, heads, dim, dtype):
    """Row stride of t [tokens][heads][dim], whose rows have to be contiguous."""
    if t.dtype != dtype or tuple(t.shape) != (tokens, heads, dim):
        raise ValueError(f"{what} must be a {dtype} tensor [{tokens}][{heads}][{dim}]")
    if (dim > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != dim):
        raise ValueError(f"the rows of {what} must be contiguous")
    return t.stride(0) if tokens > 1 else heads * dim


def _cache(k_cache, v_cache):
    import torch

    for t in (k_cache, v_cache):
        if t.dtype != torch.float16 or t.dim() != 4:
            raise ValueError("the caches must be float16 [pages][page_size][kv_heads][head_dim]")
        if t.shape[3] > 1 and t.stride(3) != 1:
            raise ValueError("a head's elements must be contiguous in the caches")
    # the stride of a dimension of one entry says nothing
    strides = [[t.stride(i) if t.shape[i] > 1 else 0 for i in range(3)] for t in (k_cache, v_cache)]
    if k_cache.shape != v_cache.shape or strides[0] != strides[1]:
        raise ValueError("both caches must have the same shape and strides")
    pages, size, heads, dim = k_cache.shape
    return _Cache(k_cache.data_ptr(), v_cache.data_ptr(), pages, *strides[0], size, heads, dim)


def _qcache_of(k_cache, v_cache, k_scale, v_scale, x):
    """The cache of a call whose rows x are [tokens][heads][head_dim]."""
    if x.dim() != 3:
        raise ValueError("q and the outputs must be [tokens][heads][head_dim]")
    return _qcache(k_cache, v_cache, k_scale, v_scale, x.shape[2])


def _qcache(k_cache, v_cache, k_scale, v_scale, dim):
    import torch

    for t in (k_cache, v_cache):
        if t.dtype != torch.uint8 or t.dim() != 4:
            raise ValueError("the caches must be uint8 [pages][page_size][kv_heads][bytes of a row]")
        if t.shape[3] > 1 and t.stride(3) != 1:
            raise ValueError("the bytes of a row must be contiguous in the caches")
    for t in (k_scale, v_scale):
        if t.dtype != torch.float16 or t.dim() != 5 or t.shape[4] != 2:
            raise ValueError("the scales must be float16 [pages][page_size][kv_heads][groups][2]")
        if t.stride(4) != 1 or (t.shape[3] > 1 and t.stride(3) != 2):
            raise ValueError("the pairs of a row must be contiguous in the scales")
    if k_scale.shape[:3] != k_cache.shape[:3]:
        raise ValueError("caches and scales must have the same pages, page_size and kv_heads")
    # the stride of a dimension of one entry says nothing
    at = [[t.stride(i) if t.shape[i] > 1 else 0 for i in range(3)]
          for t in (k_cache, v_cache, k_scale, v_scale)]
    if k_cache.shape != v_cache.shape or k_scale.shape != v_scale.shape or at[0] != at[1] or at[2] != at[3]:
        raise ValueError("keys and values must have the same shapes and strides")
    if any(s % 2 for s in at[2]):
        raise ValueError("the strides of the scales must be whole pairs")
    pages, size, heads, width = k_cache.shape
    groups = k_scale.shape[3]
    if groups == 0 or dim == 0 or dim % groups or width * 8 % dim:
        raise ValueError("rows and scales do not fit head_dim")
    return _QCache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                   pages, *at[0], *(s // 2 for s in at[2]), size, heads, dim, width * 8 // dim,
                   dim // groups)


def _append_args(struct, cache, q, k, v, cos, sin, positions, slots, q_out, interleaved):
    """The arguments of an append call, into either cache."""
    import torch

    if q.dim() != 3:
        raise ValueError("q must be [tokens][heads][head_dim]")
    tokens, heads, dim = q.shape
    if dim != cache.head_dim:
        raise ValueError("q and the caches must have the same head_dim")
    for t in (cos, sin):
        if t.dtype != torch.float32 or t.dim() != 2 or not t.is_contiguous():
            raise ValueError("cos and sin must be contiguous float32 [table_len][rot / 2]")
    if cos.shape != sin.shape:
        raise ValueError("cos and sin must have the same shape")
    code = _dtype_code(q)
    strides = [_heads("q", q, tokens, heads, dim, q.dtype),
               _heads("k", k, tokens, cache.kv_heads, dim, q.dtype),
               _heads("v", v, tokens, cache.kv_heads, dim, q.dtype),
               _heads("q_out", q_out, tokens, heads, dim, q.dtype)]
    return struct(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), cos.data_ptr(),
        sin.data_ptr(), _ints("positions", positions, tokens), _ints("slots", slots, tokens),
        cache, *strides, tokens, heads, 2 * cos.shape[1], cos.shape[0],
        int(bool(interleaved)), code)


def _attend_args(struct, cache, q, table, lens, out, scale, max_len, rows):
    """The arguments of an attention call, over either cache."""
    if q.dim() != 3:
        raise ValueError("q must be [queries][heads][head_dim]")
    n, heads, dim = q.shape
    if dim != cache.head_dim:
        raise ValueError("q and the caches must have the same head_dim")
    at, max_pages, stride = _table(table)
    if rows is None and table.shape[0] < n:
        raise ValueError("without rows, table must have a row for each query")
    code = _dtype_code(q)
    room = min(max_pages * cache.page_size, _INT32_MAX)
    if max_len is not None and max_len < 0:
        raise ValueError("max_len must not be negative")
    return struct(
        q.data_ptr(), out.data_ptr(), at, None if rows is None else _ints("rows", rows, n),
        _ints("lens", lens, n), cache,
        _heads("q", q, n, heads, dim, q.dtype), _heads("out", out, n, heads, dim, q.dtype),
        stride, n, table.shape[0], heads, max_pages,
        room if max_len is None else min(max_len, room), code,
        dim ** -0.5 if scale is None else scale)


def _scratch(name, args):
    n = ctypes.c_size_t(0)
    st = getattr(lib(), name)(ctypes.byref(args), ctypes.byref(n))
    if st != OK:
        raise SeedLMError(st, name)
    return n.value


class _Call:
    """A marshalled call: fn(*args, stream)."""

    def _set(self, name, fn, args, keep, device, stream):
        self._name, self._fn, self._args, self._keep = name, fn, args, keep
        self._device = device
        self._stream = None if stream is None else _stream_ptr(stream)

    def __call__(self, stream=None):
        """Run on `stream` (default: the one given at construction, else torch's
        current stream), with the tensors' device current."""
        import torch

        if torch.cuda.current_device() != self._device:
            raise ValueError("the tensors' device must be the current one")
        sp = _stream_ptr(stream) if stream is not None or self._stream is None else self._stream
        st = self._fn(*self._args, sp)
        if st != OK:
            raise SeedLMError(st, self._name)


class CachePlanCall(_Call):
    """One serving step's page tables, positions and slots (seedlm_cache_plan).

    lens, fresh, lens_out, ok: int32 [requests]; table: int32 [requests][max_pages]; ring:
    int32 [pages of the cache]; ring_state, ring_state_out: int32 [2]; offsets: int32
    [requests + 1]; rows, positions, slots and, where wanted, spans: int32 [tokens].  lens_out
    may be lens and ring_state_out ring_state."""

    def __init__(self, lens, fresh, table, ring, ring_state, page_size, lens_out,
                 ring_state_out, offsets, rows, positions, slots, ok, stream=None, spans=None):
        keep = (lens, fresh, table, ring, ring_state, lens_out, ring_state_out, offsets, rows,
                positions, slots, ok) + (() if spans is None else (spans,))
        device = _on_device(keep)
        n, tokens = lens.numel(), rows.numel()
        if table.shape[0] != n:
            raise ValueError("table must have a row for each request")
        if not 0 < page_size <= _INT32_MAX:
            raise ValueError("page_size must be positive and fit 32 bits")
        at, max_pages, stride = _table(table)
        args = _PlanArgs(
            _ints("lens", lens, n), _ints("fresh", fresh, n), at,
            _ints("ring", ring, ring.numel()), _ints("ring_state", ring_state, 2),
            _ints("lens_out", lens_out, n), _ints("ring_state_out", ring_state_out, 2),
            _ints("offsets", offsets, n + 1), _ints("rows", rows, tokens),
            _ints("positions", positions, tokens), _ints("slots", slots, tokens),
            _ints("ok", ok, n), None if spans is None else _ints("spans", spans, tokens), stride, n,
            page_size, max_pages, ring.numel(), tokens)
        self._set("seedlm_cache_plan", lib().seedlm_cache_plan, (ctypes.byref(args),), keep,
                  device, stream)


class CacheAppendCall(_Call):
    """Rotary positions on q and k, q_out, and k and v into their cache slots
    (seedlm_cache_append).

    q, q_out: [tokens][heads][head_dim]; k, v: [tokens][kv_heads][head_dim], float16 or
    float32, their rows contiguous; cos, sin: float32 [table_len][rot / 2]; positions, slots:
    int32 [tokens]; k_cache, v_cache: float16 [pages][page_size][kv_heads][head_dim] with any
    strides but the last.  q_out may be q."""

    def __init__(self, q, k, v, cos, sin, positions, slots, q_out, k_cache, v_cache,
                 interleaved=False, stream=None):
        keep = (q, k, v, cos, sin, positions, slots, q_out, k_cache, v_cache)
        device = _on_device(keep)
        args = _append_args(_AppendArgs, _cache(k_cache, v_cache), q, k, v, cos, sin, positions,
                            slots, q_out, interleaved)
        self._set("seedlm_cache_append", lib().seedlm_cache_append, (ctypes.byref(args),), keep,
                  device, stream)


class CacheAttendCall(_Call):
    """Attention of query tokens over their requests' pages (seedlm_cache_attend).

    q, out: [queries][heads][head_dim], float16 or float32, their rows contiguous; k_cache,
    v_cache: as for CacheAppendCall; table: int32 [table_rows][max_pages]; rows: int32
    [queries], each query's row of table (default: its own number); lens: int32 [queries],
    the tokens each query attends to, its own among them (a plan's lens_out, or its spans
    with its rows).  scale defaults to head_dim ** -0.5, max_len (the host's bound on lens)
    to what the table can hold.  out may be q."""

    def __init__(self, q, k_cache, v_cache, table, lens, out, scale=None, max_len=None,
                 stream=None, rows=None):
        keep = (q, k_cache, v_cache, table, lens, out) + (() if rows is None else (rows,))
        device = _on_device(keep)
        args = _attend_args(_AttendArgs, _cache(k_cache, v_cache), q, table, lens, out, scale,
                            max_len, rows)
        self._set("seedlm_cache_attend", lib().seedlm_cache_attend, (ctypes.byref(args),), keep,
                  device, stream)
        self._struct = args

    def scratch_bytes(self) -> int:
        """Stream scratch that the call uses."""
        return _scratch("seedlm_cache_attend_scratch_bytes", self._struct)


class QCacheAppendCall(_Call):
    """Rotary positions on q and k, q_out, and k and v quantised into their cache slots
    (seedlm_qcache_append).

    The arguments are CacheAppendCall's but for the caches: k_cache, v_cache: uint8
    [pages][page_size][kv_heads][head_dim * bits / 8], bits 4 or 8; k_scale, v_scale: float16
    [pages][page_size][kv_heads][groups][2], the (scale, offset) of each of a row's 1, 2 or 4
    groups of at least 32 elements.  Any strides but within a row, those of the caches multiples
    of 16; pools made as [pages][kv_heads][page_size][...] and transposed read fastest."""

    def __init__(self, q, k, v, cos, sin, positions, slots, q_out, k_cache, v_cache, k_scale,
                 v_scale, interleaved=False, stream=None):
        keep = (q, k, v, cos, sin, positions, slots, q_out, k_cache, v_cache, k_scale, v_scale)
        device = _on_device(keep)
        cache = _qcache_of(k_cache, v_cache, k_scale, v_scale, q)
        args = _append_args(_QAppendArgs, cache, q, k, v, cos, sin, positions, slots, q_out,
                            interleaved)
        self._set("seedlm_qcache_append", lib().seedlm_qcache_append, (ctypes.byref(args),), keep,
                  device, stream)


class QCacheReadCall(_Call):
    """What slots of a quantised cache stand for (seedlm_qcache_read).

    k_cache, v_cache, k_scale, v_scale: as for QCacheAppendCall; slots: int32 [tokens], outside
    the cache for a row of zeros; k_out, v_out: [tokens][kv_heads][head_dim], float16 or float32,
    their rows contiguous; either may be None."""

    def __init__(self, k_cache, v_cache, k_scale, v_scale, slots, k_out, v_out, stream=None):
        outs = [t for t in (k_out, v_out) if t is not None]
        if not outs:
            raise ValueError("k_out or v_out must be given")
        keep = (k_cache, v_cache, k_scale, v_scale, slots, *outs)
        device = _on_device(keep)
        cache = _qcache_of(k_cache, v_cache, k_scale, v_scale, outs[0])
        code, tokens = _dtype_code(outs[0]), slots.numel()
        strides = [0 if t is None else _heads(what, t, tokens, cache.kv_heads, cache.head_dim,
                                              outs[0].dtype)
                   for what, t in (("k_out", k_out), ("v_out", v_out))]
        args = _QReadArgs(*(None if t is None else t.data_ptr() for t in (k_out, v_out)),
                          _ints("slots", slots, tokens), cache, *strides, tokens, code)
        self._set("seedlm_qcache_read", lib().seedlm_qcache_read, (ctypes.byref(args),), keep,
                  device, stream)


class QCacheAttendCall(_Call):
    """Attention of query tokens over their requests' pages of a quantised cache
    (seedlm_qcache_attend).

    The arguments are CacheAttendCall's but for the caches, which are QCacheAppendCall's.
    Consecutive queries of one row share what they read of the cache."""

    def __init__(self, q, k_cache, v_cache, k_scale, v_scale, table, lens, out, scale=None,
                 max_len=None, stream=None, rows=None):
        keep = (q, k_cache, v_cache, k_scale, v_scale, table, lens, out) + (
            () if rows is None else (rows,))
        device = _on_device(keep)
        cache = _qcache_of(k_cache, v_cache, k_scale, v_scale, q)
        args = _attend_args(_QAttendArgs, cache, q, table, lens, out, scale, max_len, rows)
        self._set("seedlm_qcache_attend", lib().seedlm_qcache_attend, (ctypes.byref(args),), keep,
                  device, stream)
        self._struct = args

    def scratch_bytes(self) -> int:
        """Stream scratch that the call uses."""
        return _scratch("seedlm_qcache_attend_scratch_bytes", self._struct)


class LoraCall(_Call):
    """Low-rank adapters beside shared projections (seedlm_lora_many).

    sites: (x, A, B, base, y) for each projection: x [tokens][cols], base and y
    [tokens][rows] (float16 or float32, x of one type and base and y of one type over all
    sites), A float16 [adapters][rank][cols], B float16 [adapters][rows][rank], all
    contiguous; y may be base.  adapter: int32 [tokens], outside [0, adapters) for none;
    scales: float32 [adapters]."""

    def __init__(self, sites, adapter, scales, stream=None):
        import torch

        keep = (adapter, scales, *(t for site in sites for t in site))
        device = _on_device(keep)
        tokens, adapters = adapter.numel(), scales.numel()
        if scales.dtype != torch.float32 or not scales.is_contiguous():
            raise ValueError("scales must be a contiguous float32 tensor")
        structs = (_LoraSite * len(sites))()
        xdt = ydt = None
        for i, (x, A, B, base, y) in enumerate(sites):
            if not all(t.is_contiguous() for t in (x, A, B, base, y)):
                raise ValueError("the tensors of a site must be contiguous")
            if A.dim() != 3 or B.dim() != 3 or A.dtype != torch.float16 or B.dtype != torch.float16:
                raise ValueError("A and B must be float16 [adapters][rank][cols] and "
                                 "[adapters][rows][rank]")
            rank, cols, rows = A.shape[1], A.shape[2], B.shape[1]
            if A.shape[0] != adapters or B.shape[0] != adapters or B.shape[2] != rank:
                raise ValueError("A, B and scales do not fit together")
            if x.numel() != tokens * cols or base.numel() != tokens * rows or y.numel() != tokens * rows:
                raise ValueError("x must hold tokens*cols and base and y tokens*rows elements")
            xdt, ydt = xdt or x.dtype, ydt or y.dtype
            if x.dtype != xdt or y.dtype != ydt or base.dtype != ydt:
                raise ValueError("all x must share one dtype, all base and y another")
            structs[i] = _LoraSite(x.data_ptr(), A.data_ptr(), B.data_ptr(), base.data_ptr(),
                                   y.data_ptr(), rows, cols, rank)
        n = len(sites)
        codes = (_dtype_code(sites[0][0]), _dtype_code(sites[0][4])) if n else (0, 0)
        # the array rides along in the cast pointer's _objects, so it stays alive
        self._sites = ctypes.cast(structs, _vp)
        self._set("seedlm_lora_many", lib().seedlm_lora_many,
                  (self._sites, n, _ints("adapter", adapter, tokens), scales.data_ptr(), tokens,
                   adapters, *codes), keep, device, stream)

    def scratch_bytes(self) -> int:
        """Stream scratch that the call uses."""
        out = ctypes.c_size_t(0)
        sites, n, _, _, tokens, adapters, xdt, ydt = self._args
        st = lib().seedlm_lora_scratch_bytes(sites, n, tokens, adapters, xdt, ydt,
                                             ctypes.byref(out))
        if st != OK:
            raise SeedLMError(st, "seedlm_lora_scratch_bytes")
        return out.value


def seedlm_cache_plan(lens, fresh, table, ring, ring_state, page_size, lens_out, ring_state_out,
                      offsets, rows, positions, slots, ok, stream=None, spans=None):
    """One call of CachePlanCall; returns (offsets, rows, positions, slots, ok)."""
    CachePlanCall(lens, fresh, table, ring, ring_state, page_size, lens_out, ring_state_out,
                  offsets, rows, positions, slots, ok, stream, spans)()
    return offsets, rows, positions, slots, ok


def seedlm_cache_append(q, k, v, cos, sin, positions, slots, q_out, k_cache, v_cache,
                        interleaved=False, stream=None):
    """One call of CacheAppendCall; returns q_out."""
    CacheAppendCall(q, k, v, cos, sin, positions, slots, q_out, k_cache, v_cache, interleaved,
                    stream)()
    return q_out


def seedlm_cache_attend(q, k_cache, v_cache, table, lens, out, scale=None, max_len=None,
                        stream=None, rows=None):
    """One call of CacheAttendCall; returns out."""
    CacheAttendCall(q, k_cache, v_cache, table, lens, out, scale, max_len, stream, rows)()
    return out


def seedlm_qcache_append(q, k, v, cos, sin, positions, slots, q_out, k_cache, v_cache, k_scale,
                         v_scale, interleaved=False, stream=None):
    """One call of QCacheAppendCall; returns q_out."""
    QCacheAppendCall(q, k, v, cos, sin, positions, slots, q_out, k_cache, v_cache, k_scale, v_scale,
                     interleaved, stream)()
    return q_out


def seedlm_qcache_read(k_cache, v_cache, k_scale, v_scale, slots, k_out, v_out, stream=None):
    """One call of QCacheReadCall; returns (k_out, v_out)."""
    QCacheReadCall(k_cache, v_cache, k_scale, v_scale, slots, k_out, v_out, stream)()
    return k_out, v_out


def seedlm_qcache_attend(q, k_cache, v_cache, k_scale, v_scale, table, lens, out, scale=None,
                         max_len=None, stream=None, rows=None):
    """One call of QCacheAttendCall; returns out."""
    QCacheAttendCall(q, k_cache, v_cache, k_scale, v_scale, table, lens, out, scale, max_len, stream,
                     rows)()
    return out


def seedlm_lora_many(sites, adapter, scales, stream=None):
    """One call of LoraCall; returns the ys."""
    LoraCall(sites, adapter, scales, stream)()
    return [site[4] for site in sites]
