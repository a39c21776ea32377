"""The quantised cache's argument checks at the C ABI and in the binding (no GPU is touched: every
call here is refused, or does nothing)."""
import ctypes

import pytest


def _mod():
    import prng_seeded_decode_amd as S
    from prng_seeded_decode_amd import _serve

    return S, _serve


P = 4096  # an aligned address that is never used


def cache(V, **kw):
    # 64 dimensions, 4 bits, two groups, token-major
    c = V._QCache(P, P, P, P, 10, 16 * 2 * 32, 2 * 32, 32, 16 * 2 * 2, 2 * 2, 2, 16, 2, 64, 4, 32)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def append(V, c=None, **kw):
    a = V._QAppendArgs(*([P] * 8), c or cache(V), 256, 128, 128, 256, 3, 4, 64, 9, 0, 1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def read(V, c=None, **kw):
    a = V._QReadArgs(P, P, P, c or cache(V), 128, 128, 3, 1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attend(V, c=None, **kw):
    a = V._QAttendArgs(P, P, P, None, P, c or cache(V), 256, 256, 8, 3, 3, 4, 8, 100, 1, 0.1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


GEOMETRY = [
    *[({k: None}, "E_INVALID") for k in ("k", "v", "k_scale", "v_scale")],
    *[({k: 0}, "E_INVALID") for k in ("pages", "page_size", "kv_heads", "head_dim", "group")],
    *[({k: -16}, "E_INVALID") for k in ("page_stride", "token_stride", "head_stride",
                                        "scale_page_stride", "scale_token_stride",
                                        "scale_head_stride")],
    ({"pages": 2 ** 28}, "E_UNSUPPORTED"), ({"kv_heads": 16385}, "E_UNSUPPORTED"),
    ({"head_dim": 96}, "E_UNSUPPORTED"), ({"head_dim": 512}, "E_UNSUPPORTED"),
    ({"bits": 2}, "E_UNSUPPORTED"), ({"bits": 0}, "E_UNSUPPORTED"), ({"bits": -4}, "E_UNSUPPORTED"),
    ({"group": 16}, "E_UNSUPPORTED"), ({"group": 48}, "E_UNSUPPORTED"),
    ({"group": 128}, "E_UNSUPPORTED"),
    ({"head_dim": 256, "group": 32, "head_stride": 128}, "E_UNSUPPORTED"),
    ({"k": P + 8}, "E_UNSUPPORTED"), ({"v": P + 1}, "E_UNSUPPORTED"),
    ({"k_scale": P + 4}, "E_UNSUPPORTED"), ({"v_scale": P + 2}, "E_UNSUPPORTED"),
    ({"page_stride": 1032}, "E_UNSUPPORTED"), ({"token_stride": 72}, "E_UNSUPPORTED"),
    ({"head_stride": 40}, "E_UNSUPPORTED"), ({"scale_page_stride": 65}, "E_UNSUPPORTED"),
    ({"scale_token_stride": 5}, "E_UNSUPPORTED"), ({"scale_head_stride": 3}, "E_UNSUPPORTED"),
    ({"page_stride": 2 ** 36}, "E_UNSUPPORTED"), ({"token_stride": 2 ** 62}, "E_UNSUPPORTED"),
    ({"head_stride": 2 ** 35}, "E_UNSUPPORTED"), ({"scale_page_stride": 2 ** 33}, "E_UNSUPPORTED"),
    ({"scale_token_stride": 2 ** 62}, "E_UNSUPPORTED"),
    ({"scale_head_stride": 2 ** 32}, "E_UNSUPPORTED"),
    # each below its own bound, their sum above
    ({"page_stride": 2 ** 36 // 10 // 16 * 16 - 16, "token_stride": 2 ** 32 - 16}, "E_UNSUPPORTED"),
]


@pytest.mark.parametrize("c,status", GEOMETRY)
def test_every_call_refuses_a_cache_that_the_kernels_do_not_take(c, status):
    S, V = _mod()
    L = S.lib()
    want, n = getattr(S, status), ctypes.c_size_t(0)
    # strides that hold any head_dim here, so that the cache alone is refused
    a = append(V, cache(V, **c), q_stride=2048, k_stride=2048, v_stride=2048, q_out_stride=2048)
    assert L.seedlm_qcache_append(ctypes.byref(a), None) == want
    a = read(V, cache(V, **c), k_stride=2048, v_stride=2048)
    assert L.seedlm_qcache_read(ctypes.byref(a), None) == want
    a = attend(V, cache(V, **c), q_stride=2048, out_stride=2048)
    assert L.seedlm_qcache_attend(ctypes.byref(a), None) == want
    assert L.seedlm_qcache_attend_scratch_bytes(ctypes.byref(a), ctypes.byref(n)) == want


@pytest.mark.parametrize("change,status", [
    *[({k: None}, "E_INVALID") for k in ("q", "k", "v", "q_out", "positions", "slots", "cos", "sin")],
    ({"x_dtype": 2}, "E_UNSUPPORTED"), ({"tokens": -1}, "E_INVALID"), ({"heads": 0}, "E_INVALID"),
    ({"rot": 66}, "E_INVALID"), ({"rot": -2}, "E_INVALID"), ({"rot": 31}, "E_UNSUPPORTED"),
    ({"q_stride": 255}, "E_INVALID"), ({"k_stride": 127}, "E_INVALID"), ({"v_stride": 0}, "E_INVALID"),
    ({"q_out_stride": 264}, "E_INVALID"), ({"q": P + 1}, "E_INVALID"), ({"slots": P + 2}, "E_INVALID"),
    ({"tokens": 2 ** 24}, "E_UNSUPPORTED"), ({"table_len": -1}, "E_INVALID"),
    ({"heads": 16385, "q_stride": 2 ** 21, "q_out_stride": 2 ** 21}, "E_UNSUPPORTED"),
    ({"tokens": 0}, "OK"),
])
def test_append_refuses(change, status):
    S, V = _mod()
    a = append(V, **change)
    assert S.lib().seedlm_qcache_append(ctypes.byref(a), None) == getattr(S, status)


@pytest.mark.parametrize("change,status", [
    ({"slots": None}, "E_INVALID"), ({"k_out": None, "v_out": None}, "E_INVALID"),
    ({"y_dtype": 2}, "E_UNSUPPORTED"), ({"tokens": -1}, "E_INVALID"),
    ({"tokens": 2 ** 24}, "E_UNSUPPORTED"), ({"k_stride": 127}, "E_INVALID"),
    ({"v_stride": 127}, "E_INVALID"), ({"k_out": P + 1}, "E_INVALID"), ({"slots": P + 1}, "E_INVALID"),
    ({"tokens": 0, "slots": None}, "OK"), ({"tokens": 0, "k_out": None, "k_stride": 0}, "OK"),
])
def test_read_refuses(change, status):
    S, V = _mod()
    a = read(V, **change)
    assert S.lib().seedlm_qcache_read(ctypes.byref(a), None) == getattr(S, status)


@pytest.mark.parametrize("change,status", [
    *[({k: None}, "E_INVALID") for k in ("q", "out", "table", "lens")],
    ({"x_dtype": -1}, "E_UNSUPPORTED"), ({"queries": 0}, "E_INVALID"), ({"queries": 4097}, "E_INVALID"),
    ({"table_rows": 2}, "E_INVALID"), ({"table_rows": 0, "rows": P}, "E_INVALID"),
    ({"rows": P + 2}, "E_INVALID"), ({"heads": 3}, "E_INVALID"), ({"max_pages": 0}, "E_INVALID"),
    ({"max_len": -1}, "E_INVALID"), ({"table_stride": 7}, "E_INVALID"), ({"q_stride": 255}, "E_INVALID"),
    ({"out_stride": 264}, "E_INVALID"), ({"q": P + 8}, "E_UNSUPPORTED"),
    ({"q_stride": 260, "out": 2 * P}, "E_UNSUPPORTED"), ({"scale": float("nan")}, "E_INVALID"),
    ({"scale": float("inf")}, "E_INVALID"),
    ({"max_pages": 2 ** 27, "table_stride": 2 ** 27, "max_len": 2 ** 31 - 1}, "E_UNSUPPORTED"),
])
def test_attend_refuses(change, status):
    S, V = _mod()
    a, n = attend(V, **change), ctypes.c_size_t(0)
    assert S.lib().seedlm_qcache_attend(ctypes.byref(a), None) == getattr(S, status)
    assert S.lib().seedlm_qcache_attend_scratch_bytes(ctypes.byref(a), ctypes.byref(n)) == getattr(S, status)


def test_null_argument_blocks():
    S, V = _mod()
    L = S.lib()
    for fn in (L.seedlm_qcache_append, L.seedlm_qcache_read, L.seedlm_qcache_attend):
        assert fn(None, None) == S.E_INVALID
    a = attend(V)
    assert L.seedlm_qcache_attend_scratch_bytes(ctypes.byref(a), None) == S.E_INVALID


def test_the_bindings_view_of_a_cache():
    torch = pytest.importorskip("torch")
    _, V = _mod()
    codes = torch.zeros(3, 2, 16, 64, dtype=torch.uint8).transpose(1, 2)     # head-major, 4 bits
    pairs = torch.zeros(3, 2, 16, 2, 2, dtype=torch.float16).transpose(1, 2)
    c = V._qcache(codes, codes, pairs, pairs, 128)
    assert (c.pages, c.page_stride, c.token_stride, c.head_stride) == (3, 2048, 64, 1024)
    assert (c.scale_page_stride, c.scale_token_stride, c.scale_head_stride) == (64, 2, 32)
    assert (c.page_size, c.kv_heads, c.head_dim, c.bits, c.group) == (16, 2, 128, 4, 64)
    bad = [
        (codes.half(), codes, pairs, pairs, 128), (codes, codes[:2], pairs, pairs, 128),
        (codes, codes.contiguous(), pairs, pairs, 128), (codes, codes, pairs.float(), pairs, 128),
        (codes, codes, pairs, pairs.contiguous(), 128), (codes, codes, pairs[:2], pairs[:2], 128),
        (codes, codes, pairs[..., 0], pairs[..., 0], 128), (codes, codes, pairs, pairs, 96),
        (codes, codes, pairs.transpose(3, 4), pairs.transpose(3, 4), 128),
        (codes[..., ::2], codes[..., ::2], pairs, pairs, 128),
    ]
    for args in bad:
        with pytest.raises(ValueError):
            V._qcache(*args)


def test_python_wrappers_refuse_what_does_not_fit():
    torch = pytest.importorskip("torch")
    S, _ = _mod()
    q = torch.zeros(2, 4, 64, dtype=torch.float16)
    c, p = torch.zeros(3, 16, 2, 32, dtype=torch.uint8), torch.zeros(3, 16, 2, 1, 2, dtype=torch.float16)
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # host tensors
        S.seedlm_qcache_attend(q, c, c, p, p, ints.view(2, 1), ints, q)
    with pytest.raises(ValueError):
        S.seedlm_qcache_read(c, c, p, p, ints, None, None)
