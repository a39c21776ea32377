"""seedlm_cache_append against the rotation in 64 bits, within two fp32 roundings and the
output's own (tolerances of serve_ref)."""
import numpy as np
import pytest

import serve_ref as R

pytestmark = pytest.mark.gpu


def make(seed, tokens, heads, kv, dim, rot, f16, size, pages, table_len=97):
    rng = np.random.default_rng(seed)
    dt = np.float16 if f16 else np.float32
    x = {k: rng.standard_normal((tokens, h, dim)).astype(dt)
         for k, h in (("q", heads), ("k", kv), ("v", kv))}
    angle = rng.uniform(0, 6.28, (table_len, rot // 2))
    x["cos"], x["sin"] = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    x["positions"] = rng.integers(0, table_len, tokens)
    x["slots"] = rng.permutation(size * pages)[:tokens]
    for k in ("k_cache", "v_cache"):
        x[k] = rng.standard_normal((pages, size, kv, dim)).astype(np.float16)
    return x


def expected(x, interleaved):
    f16 = x["q"].dtype == np.float16
    pages, size = x["k_cache"].shape[:2]
    pos, slot = x["positions"], x["slots"]
    turns = (pos >= 0) & (pos < x["cos"].shape[0])
    p = np.where(turns, pos, 0)
    q, qt = R.rotate(x["q"], x["cos"][p], x["sin"][p], interleaved)
    k, kt = R.rotate(x["k"], x["cos"][p], x["sin"][p], interleaved)
    q[~turns], qt[~turns] = 0, 0
    # elements that do not turn are copied
    qt += np.where(qt > 0, R.rounding(q, f16), 0)
    kc, vc = x["k_cache"].astype(np.float64), x["v_cache"].astype(np.float64)
    kct, vct = np.zeros(kc.shape), np.zeros(vc.shape)
    for t in np.nonzero(turns & (slot >= 0) & (slot < pages * size))[0]:
        at = slot[t] // size, slot[t] % size
        kc[at], vc[at] = k[t], x["v"][t].astype(np.float64)
        kct[at] = kt[t] + R.rounding(k[t], True)
        vct[at] = 0 if f16 else R.rounding(vc[at], True)
    return (q, qt), (kc, kct), (vc, vct)


def device(x, head_major=False, pad=0):
    import torch

    d = {}
    for name, a in x.items():
        if name in ("positions", "slots"):
            d[name] = torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
        elif name in ("k_cache", "v_cache"):
            t = torch.from_numpy(a).cuda()
            if head_major:
                t = t.transpose(1, 2).contiguous().transpose(1, 2)
            d[name] = t
        elif name in "qkv" and pad:
            t = torch.zeros((a.shape[0], a.shape[1] * a.shape[2] + pad), device="cuda",
                            dtype=torch.from_numpy(a).dtype)
            view = t[:, : a.shape[1] * a.shape[2]].view(a.shape)
            view.copy_(torch.from_numpy(a))
            d[name] = view
        else:
            d[name] = torch.from_numpy(a).cuda()
    return d


def check(x, interleaved, head_major=False, pad=0, in_place=False):
    import torch

    import prng_seeded_decode_amd as S

    d = device(x, head_major, pad)
    q_out = d["q"] if in_place else torch.full(x["q"].shape, 7.0, dtype=d["q"].dtype, device="cuda")
    S.seedlm_cache_append(d["q"], d["k"], d["v"], d["cos"], d["sin"], d["positions"], d["slots"],
                          q_out, d["k_cache"], d["v_cache"], interleaved=interleaved)
    torch.cuda.synchronize()
    for got, (ref, tol) in zip((q_out, d["k_cache"], d["v_cache"]), expected(x, interleaved)):
        err = np.abs(got.double().cpu().numpy() - ref)
        assert np.all(err <= tol), (err - tol).max()


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,kv,dim,rot,size,pages,head_major,pad", [
    (1, 1, 1, 64, 64, 16, 1, False, 0),
    (3, 32, 8, 128, 128, 16, 4, False, 0),
    (17, 64, 8, 128, 64, 24, 3, True, 0),
    (5, 4, 2, 256, 256, 1, 9, False, 64),
    (129, 40, 10, 64, 32, 16, 12, True, 32),
    (7, 3, 1, 6, 4, 5, 3, False, 0),       # units of one pair
    (9, 5, 5, 80, 20, 16, 2, True, 0),
    (4, 2, 2, 512, 510, 4, 2, False, 3),
    (6, 4, 2, 128, 0, 16, 2, False, 0),    # nothing turns
])
def test_append_matches_64_bits(tokens, heads, kv, dim, rot, size, pages, head_major, pad, f16,
                                interleaved):
    x = make([tokens, heads, dim, rot], tokens, heads, kv, dim, rot, f16, size, pages)
    check(x, interleaved, head_major, pad)
    check(x, interleaved, head_major, pad, in_place=True)


@pytest.mark.parametrize("dim", [128, 10])
def test_append_padding_rows_write_nothing(dim):
    x = make([1, dim], 12, 4, 2, dim, dim, True, 16, 4)
    x["slots"][[0, 5]] = [-1, 64]          # no slot, a slot past the cache
    x["slots"][7] = -2 ** 31
    x["positions"][[2, 9]] = [-1, 97]      # positions outside the table
    check(x, False)
    x["slots"][:] = -1
    check(x, True)


def test_append_carries_infinities_and_nan_to_their_own_elements_only():
    import torch

    import prng_seeded_decode_amd as S

    x = make([5], 6, 4, 2, 128, 128, True, 16, 2)
    bad = {k: x[k].copy() for k in "qkv"}
    bad["q"][1, 2, 5], bad["k"][2, 1, 70], bad["v"][3, 0, 9] = np.nan, np.inf, -np.inf
    outs = []
    for src in (x, dict(x, **bad)):
        d = device(src)
        q_out = torch.zeros_like(d["q"])
        S.seedlm_cache_append(d["q"], d["k"], d["v"], d["cos"], d["sin"], d["positions"],
                              d["slots"], q_out, d["k_cache"], d["v_cache"])
        outs.append([t.cpu().numpy() for t in (q_out, d["k_cache"], d["v_cache"])])
    for clean, dirty in zip(*outs):
        assert np.array_equal(clean[np.isfinite(dirty)], dirty[np.isfinite(dirty)])
    assert [(~np.isfinite(t)).sum() for t in outs[1]] == [2, 2, 1]


def test_append_of_no_tokens():
    import torch

    import prng_seeded_decode_amd as S

    x = make([2], 1, 4, 2, 64, 64, True, 16, 2)
    d = device(x)
    e = {k: d[k][:0] for k in ("q", "k", "v", "positions", "slots")}
    before = d["k_cache"].clone()
    S.seedlm_cache_append(e["q"], e["k"], e["v"], d["cos"], d["sin"], e["positions"], e["slots"],
                          e["q"].clone(), d["k_cache"], d["v_cache"])
    torch.cuda.synchronize()
    assert torch.equal(before, d["k_cache"])
