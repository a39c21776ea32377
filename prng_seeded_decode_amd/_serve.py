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
        import torch

        keep = (q, k, v, cos, sin, positions, slots, q_out, k_cache, v_cache)
        device = _on_device(keep)
        cache = _cache(k_cache, v_cache)
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
        args = _AppendArgs(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), cos.data_ptr(),
            sin.data_ptr(), _ints("positions", positions, tokens), _ints("slots", slots, tokens),
            cache, *strides, tokens, heads, 2 * cos.shape[1], cos.shape[0],
            int(bool(interleaved)), code)
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
        cache = _cache(k_cache, v_cache)
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
        args = _AttendArgs(
            q.data_ptr(), out.data_ptr(), at, None if rows is None else _ints("rows", rows, n),
            _ints("lens", lens, n), cache,
            _heads("q", q, n, heads, dim, q.dtype), _heads("out", out, n, heads, dim, q.dtype),
            stride, n, table.shape[0], heads, max_pages,
            room if max_len is None else min(max_len, room), code,
            dim ** -0.5 if scale is None else scale)
        self._set("seedlm_cache_attend", lib().seedlm_cache_attend, (ctypes.byref(args),), keep,
                  device, stream)
        self._struct = args

    def scratch_bytes(self) -> int:
        """Stream scratch that the call uses."""
        n = ctypes.c_size_t(0)
        st = lib().seedlm_cache_attend_scratch_bytes(ctypes.byref(self._struct), ctypes.byref(n))
        if st != OK:
            raise SeedLMError(st, "seedlm_cache_attend_scratch_bytes")
        return n.value


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


def seedlm_lora_many(sites, adapter, scales, stream=None):
    """One call of LoraCall; returns the ys."""
    LoraCall(sites, adapter, scales, stream)()
    return [site[4] for site in sites]
