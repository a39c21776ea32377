"""The serving operators' argument checks at the C ABI (no GPU is touched: every call here is
refused, or does nothing)."""
import ctypes

import pytest


def _mod():
    import prng_seeded_decode_amd as S
    from prng_seeded_decode_amd import _serve

    return S, _serve


P = 4096  # an aligned address that is never used


def plan(V, **kw):
    a = V._PlanArgs(*([P] * 12), None, 8, 4, 16, 8, 100, 32)
    a.lens_out, a.ring_state_out = 2 * P, 2 * P
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def cache(V, **kw):
    c = V._Cache(P, P, 10, 16 * 2 * 64, 2 * 64, 64, 16, 2, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def append(V, c=None, **kw):
    a = V._AppendArgs(*([P] * 8), c or cache(V), 256, 128, 128, 256, 3, 4, 64, 9, 0, 1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attend(V, c=None, **kw):
    a = V._AttendArgs(P, P, P, None, P, c or cache(V), 256, 256, 8, 3, 3, 4, 8, 100, 1, 0.1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    *[({k: None}, "E_INVALID") for k in ("lens", "fresh", "table", "ring", "ring_state",
                                         "lens_out", "ring_state_out", "offsets", "rows",
                                         "positions", "slots", "ok")],
    ({"requests": 0}, "E_INVALID"), ({"requests": 4097}, "E_INVALID"),
    ({"page_size": 0}, "E_INVALID"), ({"max_pages": 0}, "E_INVALID"), ({"pool": 0}, "E_INVALID"),
    ({"tokens": -1}, "E_INVALID"), ({"table_stride": 7}, "E_INVALID"),
    ({"spans": P + 1}, "E_INVALID"), ({"lens": P + 2}, "E_INVALID"), ({"lens_out": P + 4}, "E_INVALID"),
    ({"lens_out": P - 8}, "E_INVALID"), ({"ring_state_out": P + 4}, "E_INVALID"),
    ({"max_pages": 2 ** 27, "table_stride": 2 ** 27}, "E_UNSUPPORTED"),
    ({"pool": 2 ** 27}, "E_UNSUPPORTED"), ({"tokens": 2 ** 30 + 1}, "E_UNSUPPORTED"),
    ({"pool": 2 ** 30 + 1, "page_size": 1}, "E_UNSUPPORTED"),
])
def test_plan_refuses(change, status):
    S, V = _mod()
    a = plan(V, **change)
    assert S.lib().seedlm_cache_plan(ctypes.byref(a), None) == getattr(S, status)


@pytest.mark.parametrize("c,change,status", [
    ({"k": None}, {}, "E_INVALID"), ({"v": P + 1}, {}, "E_INVALID"), ({"pages": 0}, {}, "E_INVALID"),
    ({"page_size": 0}, {}, "E_INVALID"), ({"kv_heads": 0}, {}, "E_INVALID"),
    ({"head_dim": 0}, {}, "E_INVALID"), ({"token_stride": -64}, {}, "E_INVALID"),
    ({"pages": 2 ** 28}, {}, "E_UNSUPPORTED"), ({"head_dim": 63}, {"rot": 0}, "E_UNSUPPORTED"),
    *[({}, {k: None}, "E_INVALID") for k in ("q", "k", "v", "q_out", "positions", "slots", "cos",
                                             "sin")],
    ({}, {"x_dtype": 2}, "E_UNSUPPORTED"), ({}, {"tokens": -1}, "E_INVALID"),
    ({}, {"heads": 0}, "E_INVALID"), ({}, {"rot": 66}, "E_INVALID"), ({}, {"rot": -2}, "E_INVALID"),
    ({}, {"rot": 31}, "E_UNSUPPORTED"), ({}, {"q_stride": 255}, "E_INVALID"),
    ({}, {"k_stride": 127}, "E_INVALID"), ({}, {"v_stride": 0}, "E_INVALID"),
    ({}, {"q_out_stride": 264}, "E_INVALID"), ({}, {"q": P + 1}, "E_INVALID"),
    ({}, {"tokens": 2 ** 24}, "E_UNSUPPORTED"), ({}, {"table_len": -1}, "E_INVALID"),
    ({"head_dim": 514}, {}, "E_UNSUPPORTED"),
    ({}, {"heads": 16385, "q_stride": 2 ** 21, "q_out_stride": 2 ** 21}, "E_UNSUPPORTED"),
])
def test_append_refuses(c, change, status):
    S, V = _mod()
    a = append(V, cache(V, **c), **change)
    assert S.lib().seedlm_cache_append(ctypes.byref(a), None) == getattr(S, status)


@pytest.mark.parametrize("c,change,status", [
    ({"k": None}, {}, "E_INVALID"), ({"pages": 0}, {}, "E_INVALID"),
    ({"k": P + 8}, {}, "E_UNSUPPORTED"), ({"page_stride": 2052}, {}, "E_UNSUPPORTED"),
    ({"token_stride": 129}, {}, "E_UNSUPPORTED"), ({"head_stride": 65}, {}, "E_UNSUPPORTED"),
    ({"head_dim": 96}, {"q_stride": 400, "out_stride": 400}, "E_UNSUPPORTED"),
    ({"page_stride": 2 ** 34}, {}, "E_UNSUPPORTED"), ({"token_stride": 2 ** 33}, {}, "E_UNSUPPORTED"),
    ({"head_stride": 2 ** 35}, {}, "E_UNSUPPORTED"),
    *[({}, {k: None}, "E_INVALID") for k in ("q", "out", "table", "lens")],
    ({}, {"x_dtype": -1}, "E_UNSUPPORTED"), ({}, {"queries": 0}, "E_INVALID"),
    ({}, {"queries": 4097}, "E_INVALID"), ({}, {"table_rows": 2}, "E_INVALID"),
    ({}, {"table_rows": 0, "rows": P}, "E_INVALID"), ({}, {"rows": P + 2}, "E_INVALID"), ({}, {"heads": 3}, "E_INVALID"),
    ({}, {"max_pages": 0}, "E_INVALID"), ({}, {"max_len": -1}, "E_INVALID"),
    ({}, {"table_stride": 7}, "E_INVALID"), ({}, {"q_stride": 255}, "E_INVALID"),
    ({}, {"out_stride": 264}, "E_INVALID"), ({}, {"q": P + 8}, "E_UNSUPPORTED"),
    ({}, {"q_stride": 260, "out": 2 * P}, "E_UNSUPPORTED"),
    ({}, {"scale": float("nan")}, "E_INVALID"), ({}, {"scale": float("inf")}, "E_INVALID"),
    ({}, {"max_pages": 2 ** 27, "table_stride": 2 ** 27, "max_len": 2 ** 31 - 1}, "E_UNSUPPORTED"),
])
def test_attend_refuses(c, change, status):
    S, V = _mod()
    a = attend(V, cache(V, **c), **change)
    n = ctypes.c_size_t(0)
    assert S.lib().seedlm_cache_attend(ctypes.byref(a), None) == getattr(S, status)
    assert S.lib().seedlm_cache_attend_scratch_bytes(ctypes.byref(a), ctypes.byref(n)) == getattr(S, status)


def test_null_argument_blocks():
    S, V = _mod()
    L = S.lib()
    for fn in (L.seedlm_cache_plan, L.seedlm_cache_append, L.seedlm_cache_attend):
        assert fn(None, None) == S.E_INVALID
    a = attend(V)
    assert L.seedlm_cache_attend_scratch_bytes(ctypes.byref(a), None) == S.E_INVALID
    assert L.seedlm_cache_append(ctypes.byref(append(V, tokens=0)), None) == S.OK


def lora(S, V, n=1, tokens=4, adapters=2, xdt=1, ydt=1, adapter=P, scales=P, **kw):
    site = V._LoraSite(P, P, P, P, P, 64, 32, 8)
    for k, v in kw.items():
        setattr(site, k, v)
    arr = (V._LoraSite * 2)(site, site)
    return S.lib().seedlm_lora_many(ctypes.cast(arr, ctypes.c_void_p), n, adapter, scales, tokens,
                                    adapters, xdt, ydt, None)


@pytest.mark.parametrize("change,status", [
    *[({k: None}, "E_INVALID") for k in ("x", "A", "B", "base", "y", "adapter", "scales")],
    ({"rows": 0}, "E_INVALID"), ({"cols": 0}, "E_INVALID"), ({"rank": 0}, "E_INVALID"),
    ({"rank": 257}, "E_INVALID"), ({"n": -1}, "E_INVALID"), ({"tokens": -1}, "E_INVALID"),
    ({"adapters": 0}, "E_INVALID"), ({"xdt": 2}, "E_UNSUPPORTED"), ({"ydt": -1}, "E_UNSUPPORTED"),
    ({"x": P + 1}, "E_INVALID"), ({"y": P + 1}, "E_INVALID"), ({"adapter": P + 2}, "E_INVALID"),
    ({"tokens": 2 ** 24}, "E_UNSUPPORTED"), ({"rows": 2 ** 24}, "E_UNSUPPORTED"),
    ({"cols": 2 ** 24}, "E_UNSUPPORTED"), ({"n": 0}, "OK"), ({"tokens": 0}, "OK"),
])
def test_lora_refuses(change, status):
    S, V = _mod()
    assert lora(S, V, **change) == getattr(S, status)


def test_lora_scratch_is_the_largest_groups():
    S, V = _mod()
    n = ctypes.c_size_t(0)
    # rank 32: no site takes the one-launch form, which needs none
    arr = (V._LoraSite * 17)(*[V._LoraSite(P, P, P, P, P, 64, 32, 32)] * 17)

    def ask(k):
        assert S.lib().seedlm_lora_scratch_bytes(ctypes.cast(arr, ctypes.c_void_p), k, 4, 2, 1, 1,
                                                 ctypes.byref(n)) == S.OK
        return n.value

    assert ask(0) == 0 and 0 < ask(1) < ask(8) == ask(17)
    assert S.lib().seedlm_lora_scratch_bytes(None, 1, 4, 2, 1, 1, ctypes.byref(n)) == S.E_INVALID
    assert S.lib().seedlm_lora_scratch_bytes(None, 0, 4, 0, 1, 1, ctypes.byref(n)) == S.E_INVALID


def test_python_wrappers_refuse_what_does_not_fit():
    torch = pytest.importorskip("torch")
    S, _ = _mod()
    q = torch.zeros(2, 4, 64, dtype=torch.float16)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.float16)
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # host tensors
        S.seedlm_cache_attend(q, c, c, ints.view(2, 1), ints, q)
    with pytest.raises(ValueError):
        S.seedlm_lora_many([(q, c, c, q, q)], ints, torch.zeros(3))
