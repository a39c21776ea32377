"""seedlm_qcache_append and seedlm_qcache_read.

The quantisation is defined in fp32 steps, each rounded, so codes and pairs have to equal the same
steps in numpy, bit by bit.  What reads back is held to the rotation in 64 bits besides: half a
step, what the step's own rounding moves a code's value by, and the roundings before."""
import numpy as np
import pytest

import qcache_ref as Q
import serve_ref as R

pytestmark = pytest.mark.gpu

U16 = R.U16


def make(seed, tokens, heads, kv, dim, rot, f16, size, pages, bits, group, table_len=97):
    rng = np.random.default_rng(seed)
    dt = np.float16 if f16 else np.float32
    x = {k: rng.standard_normal((tokens, h, dim)).astype(dt)
         for k, h in (("q", heads), ("k", kv), ("v", kv))}
    x["k"] = (x["k"] * np.where(rng.random((kv, dim)) < 0.05, 9.0, 1.0)).astype(dt)
    angle = rng.uniform(0, 6.28, (table_len, rot // 2))
    x["cos"], x["sin"] = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    x["positions"] = rng.integers(0, table_len, tokens)
    x["slots"] = rng.permutation(size * pages)[:tokens]
    for k in ("k", "v"):
        x[k + "_cache"] = rng.integers(0, 256, (pages, size, kv, dim * bits // 8)).astype(np.uint8)
        x[k + "_scale"] = rng.standard_normal((pages, size, kv, dim // group, 2)).astype(np.float16)
    return x


def device(x, head_major=False, pad=0):
    import torch

    d = {}
    for name, a in x.items():
        if name in ("positions", "slots"):
            d[name] = torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
            continue
        t = torch.from_numpy(a).cuda()
        if "cache" in name or "scale" in name:
            if head_major:
                t = t.transpose(1, 2).contiguous().transpose(1, 2)
            elif pad and "cache" in name:  # rows 16 bytes apart
                wide = torch.full((*t.shape[:3], t.shape[3] + 16), 77, dtype=t.dtype, device="cuda")
                wide[..., :-16] = t
                t = wide[..., :-16]
        elif name in "qkv" and pad:
            n = a.shape[1] * a.shape[2]
            wide = torch.zeros((a.shape[0], n + pad), device="cuda", dtype=t.dtype)
            wide[:, :n] = t.view(a.shape[0], n)
            t = wide[:, :n].view(a.shape)
        d[name] = t
    return d


CACHE = ("k_cache", "v_cache", "k_scale", "v_scale")


def live_rows(x):
    pages, size = x["k_cache"].shape[:2]
    turns = (x["positions"] >= 0) & (x["positions"] < x["cos"].shape[0])
    return turns, np.nonzero(turns & (x["slots"] >= 0) & (x["slots"] < pages * size))[0]


def expected(x, interleaved, bits, group):
    size = x["k_cache"].shape[1]
    turns, live = live_rows(x)
    p = np.where(turns, x["positions"], 0)
    out = {n: x[n].copy() for n in CACHE}
    vals = {"k": Q.rotate32(x["k"], x["cos"][p], x["sin"][p], interleaved)}
    with np.errstate(over="ignore"):
        vals["v"] = x["v"].astype(np.float16)
    for name, v in vals.items():
        rows, pairs = Q.quantise(v, bits, group)
        for t in live:
            at = x["slots"][t] // size, x["slots"][t] % size
            out[name + "_cache"][at], out[name + "_scale"][at] = rows[t], pairs[t]
    q, qt = R.rotate(x["q"], x["cos"][p], x["sin"][p], interleaved)
    q[~turns], qt[~turns] = 0, 0
    qt += np.where(qt > 0, R.rounding(q, x["q"].dtype == np.float16), 0)
    return (q, qt), out


def append(x, interleaved=False, head_major=False, pad=0, in_place=False, **kw):
    import torch

    import prng_seeded_decode_amd as S

    d = device(x, head_major, pad)
    q_out = d["q"] if in_place else torch.full(x["q"].shape, 7.0, dtype=d["q"].dtype, device="cuda")
    S.seedlm_qcache_append(d["q"], d["k"], d["v"], d["cos"], d["sin"], d["positions"], d["slots"],
                           q_out, *(d[n] for n in CACHE), interleaved=interleaved, **kw)
    torch.cuda.synchronize()
    return d, q_out


def same_bits(a, b):
    return np.array_equal(a.view(np.uint16 if a.dtype == np.float16 else a.dtype),
                          b.view(np.uint16 if b.dtype == np.float16 else b.dtype))


def check(x, bits, group, interleaved=False, **kw):
    d, q_out = append(x, interleaved, **kw)
    (q, qt), caches = expected(x, interleaved, bits, group)
    err = np.abs(q_out.double().cpu().numpy() - q)
    assert np.all(err <= qt), (err - qt).max()
    for n in CACHE:
        got = d[n].cpu().numpy()
        if got.dtype == np.float16:  # -0 and 0 are the same offset, any NaN the same scale
            assert np.array_equal(got, caches[n], equal_nan=True), n
        else:
            assert np.array_equal(got, caches[n]), n
    return d


CASES = [
    (1, 1, 1, 64, 64, 16, 1, False, 0),
    (3, 32, 8, 128, 128, 16, 4, False, 0),
    (17, 64, 8, 128, 64, 24, 3, True, 0),
    (5, 4, 2, 256, 256, 1, 9, False, 64),
    (129, 40, 10, 64, 32, 16, 12, True, 32),
    (33, 3, 3, 128, 96, 5, 7, False, 0),
    (9, 5, 5, 128, 20, 16, 2, True, 0),     # pairs that lie apart from any alignment
    (4, 2, 2, 256, 254, 4, 2, False, 3),    # rows of odd addresses
    (6, 4, 2, 128, 0, 16, 2, False, 0),     # nothing turns
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,kv,dim,rot,size,pages,head_major,pad", CASES)
def test_append_gives_the_codes_of_the_definition(tokens, heads, kv, dim, rot, size, pages, head_major,
                                                  pad, f16, interleaved, bits):
    for groups in (1, 2, 4) if dim > 64 else (1, 2):
        x = make([tokens, heads, dim, rot, bits], tokens, heads, kv, dim, rot, f16, size, pages, bits,
                 dim // groups)
        check(x, bits, dim // groups, interleaved, head_major=head_major, pad=pad)
    check(x, bits, dim // groups, interleaved, head_major=head_major, pad=pad, in_place=True)


@pytest.mark.parametrize("bits,group", [(4, 32), (4, 128), (8, 64)])
@pytest.mark.parametrize("f16", [True, False])
def test_what_reads_back_is_within_half_a_step(bits, group, f16):
    import torch

    import prng_seeded_decode_amd as S

    x = make([3, bits, group], 200, 4, 2, 128, 128, f16, 16, 20, bits, group)
    d, _ = append(x)
    outs = [torch.full((200, 2, 128), 5.0, device="cuda") for _ in range(2)]
    S.seedlm_qcache_read(*(d[n] for n in CACHE), d["slots"], *outs)
    torch.cuda.synchronize()
    k, kt = R.rotate(x["k"], x["cos"][x["positions"]], x["sin"][x["positions"]], False)
    size = 16
    for got, ref, off, pool in ((outs[0], k, kt, "k_scale"), (outs[1], x["v"].astype(np.float64), 0.0, "v_scale")):
        at = x["slots"] // size, x["slots"] % size
        s = d[pool].cpu().numpy()[at][..., 0].astype(np.float64).repeat(group, -1).reshape(ref.shape)
        # the rotation and fp16; half a step; a step that was rounded down by 2^-11 (and no less
        # than 2^-25) leaves that much of each of up to 2^bits - 1 steps to the last code
        tol = off + R.rounding(ref, True) + s / 2
        tol += (2 ** bits - 1) * np.maximum(s * U16, 2.0 ** -25) + R.U32 * np.abs(ref)
        err = np.abs(got.double().cpu().numpy() - ref)
        assert np.all(err <= tol), (err - tol).max()


@pytest.mark.parametrize("bits", [4, 8])
def test_groups_without_a_spread_and_with_small_or_large_ones(bits):
    x = make([7, bits], 8, 1, 1, 64, 0, True, 16, 1, bits, 32)
    v = x["v"]
    v[0] = 1.5                                         # s = 0
    v[1], v[1, 0, 3] = 0.0, 2.0 ** -24                 # s rounds to 0
    v[2], v[2, 0, 3] = 0.0, np.float16(2.0 ** -24 * 40)  # s below fp16's normal numbers
    v[3], v[3, 0, 3], v[3, 0, 4] = 0.0, 65504, -65504
    v[4] = -0.0
    v[5, 0, :16], v[5, 0, 16:32] = np.float16(0.5), np.float16(0.5 + 15)  # whole steps
    v[6, 0] = np.arange(64) / 2                        # ties between codes
    check(x, bits, 32)


def test_ties_and_borders_over_many_groups():
    # small whole numbers: (x - o) / s falls on halves in a large part of the elements
    for bits in (4, 8):
        x = make([8, bits], 500, 1, 4, 128, 0, True, 16, 40, bits, 32)
        rng = np.random.default_rng(2)
        for k in "kv":
            x[k] = (rng.integers(-60, 61, x[k].shape) / 2.0 ** rng.integers(0, 6, (500, 4, 1))).astype(np.float16)
        check(x, bits, 32)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_nan_and_infinities_keep_to_their_group(dim, f16):
    import torch

    import prng_seeded_decode_amd as S

    bits, group = 4, dim // 2
    x = make([9, dim], 6, 2, 2, dim, 0, f16, 16, 2, bits, group)
    x["k"][1, 1, 5], x["v"][2, 0, dim - 1], x["k"][3, 0, 0] = np.nan, np.inf, -np.inf
    if not f16:
        x["v"][4, 1, 7] = 1e6  # past fp16
    d = check(x, bits, group)
    outs = [torch.zeros((6, 2, dim), dtype=torch.float16, device="cuda") for _ in range(2)]
    S.seedlm_qcache_read(*(d[n] for n in CACHE), d["slots"], *outs)
    k, v = (t.isnan().cpu().numpy() for t in outs)
    want = np.zeros((2, 6, 2, dim), bool)
    want[0, 1, 1, :group] = want[0, 3, 0, :group] = True
    want[1, 2, 0, group:] = True
    if not f16:
        want[1, 4, 1, :group] = True
    assert np.array_equal(k, want[0]) and np.array_equal(v, want[1])


@pytest.mark.parametrize("bits,dim,rot", [(4, 128, 128), (8, 64, 10)])
def test_padding_rows_write_nothing(bits, dim, rot):
    x = make([1, dim], 12, 4, 2, dim, rot, True, 16, 4, bits, 32)
    x["slots"][[0, 5]] = [-1, 64]          # no slot, a slot past the cache
    x["slots"][7] = -2 ** 31
    x["positions"][[2, 9]] = [-1, 97]      # positions outside the table
    check(x, bits, 32)
    x["slots"][:] = -1
    check(x, bits, 32, True)


def test_append_and_read_of_no_tokens():
    import torch

    import prng_seeded_decode_amd as S

    x = make([2], 1, 4, 2, 64, 64, True, 16, 2, 4, 32)
    d = device(x)
    e = {k: d[k][:0] for k in ("q", "k", "v", "positions", "slots")}
    cache = [d[n] for n in CACHE]
    before = [t.clone() for t in cache]
    S.seedlm_qcache_append(e["q"], e["k"], e["v"], d["cos"], d["sin"], e["positions"], e["slots"],
                           e["q"].clone(), *cache)
    S.seedlm_qcache_read(*cache, e["slots"], e["k"].clone(), None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before[:2], cache[:2]))


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("bits,dim,groups,head_major,pad", [
    (4, 64, 1, False, 0), (4, 64, 2, True, 0), (4, 128, 1, True, 0), (4, 128, 4, False, 16),
    (4, 256, 2, True, 0), (8, 64, 2, False, 16), (8, 128, 1, False, 0), (8, 256, 4, True, 0)])
def test_read(bits, dim, groups, head_major, pad, f16):
    import torch

    import prng_seeded_decode_amd as S

    x = make([4, dim, bits], 1, 1, 3, dim, 0, True, 8, 30, bits, dim // groups)
    d = device({n: x[n] for n in CACHE}, head_major, pad)
    slots = np.array([5, 239, 0, -1, 240, 5, 17, 100, -2 ** 31, 2 ** 31 - 1, 200, 7, 8])
    n = len(slots)
    dt = torch.float16 if f16 else torch.float32
    wide = torch.full((n, 3 * dim + 5), 9.0, dtype=dt, device="cuda")  # rows of odd addresses
    k_out, v_out = wide[:, :3 * dim].view(n, 3, dim), torch.full((n, 3, dim), 9.0, dtype=dt, device="cuda")
    S.seedlm_qcache_read(*(d[m] for m in CACHE), torch.from_numpy(slots.astype(np.int32)).cuda(),
                         k_out, v_out)
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < 240)
    at = np.where(live, slots, 0) // 8, np.where(live, slots, 0) % 8
    for name, got in (("k", k_out), ("v", v_out)):
        ref, mag = Q.values(x[name + "_cache"][at], x[name + "_scale"][at], bits)
        ref[~live], mag[~live] = 0, 0
        # s c is exact in fp32; one rounding there, one to the output's type
        tol = R.rounding(ref, f16) + R.U32 * np.abs(ref)
        tol[~live] = 0
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)
    assert (wide[:, 3 * dim:] == 9).all()
    alone = torch.full((n, 3, dim), 9.0, dtype=dt, device="cuda")
    S.seedlm_qcache_read(*(d[m] for m in CACHE), torch.from_numpy(slots.astype(np.int32)).cuda(),
                         None, alone)
    assert torch.equal(alone, v_out)


def test_read_of_many_tokens_and_a_strided_output():
    import torch

    import prng_seeded_decode_amd as S

    x = make([5], 1, 1, 2, 128, 0, True, 16, 200, 4, 64)
    d = device({n: x[n] for n in CACHE}, True)
    slots = np.random.default_rng(0).integers(-5, 3210, 5003)
    both = torch.full((5003, 2, 2, 128), 9.0, dtype=torch.float16, device="cuda")
    S.seedlm_qcache_read(*(d[m] for m in CACHE), torch.from_numpy(slots.astype(np.int32)).cuda(),
                         both[:, 0], both[:, 1])
    got = both.double().cpu().numpy()
    live = (slots >= 0) & (slots < 3200)
    at = np.where(live, slots, 0) // 16, np.where(live, slots, 0) % 16
    for i, name in enumerate("kv"):
        ref, _ = Q.values(x[name + "_cache"][at], x[name + "_scale"][at], 4)
        ref[~live] = 0
        assert np.all(np.abs(got[:, i] - ref) <= R.rounding(ref, True) + R.U32 * np.abs(ref))


def test_offsets_past_32_bits():
    # code pools of 2^32 bytes and more; only the rows in use are ever written or read
    import torch

    import prng_seeded_decode_amd as S

    size, kv, dim = 16, 8, 256
    pages = 2 ** 32 // (size * kv * dim) + 5
    x = make([6], 40, 8, kv, dim, dim, True, size, 4, 8, 64)
    d = device(x)
    pools = {}
    for n in CACHE:
        pools[n] = torch.empty((pages, *d[n].shape[1:]), dtype=d[n].dtype, device="cuda")
        pools[n][:2], pools[n][-2:] = d[n][:2], d[n][2:]
    slots = np.where(x["slots"] < 2 * size, x["slots"], x["slots"] + (pages - 4) * size)
    d["slots"] = torch.from_numpy(slots.astype(np.int32)).cuda()
    cache = [pools[n] for n in CACHE]
    S.seedlm_qcache_append(d["q"], d["k"], d["v"], d["cos"], d["sin"], d["positions"], d["slots"],
                           d["q"].clone(), *cache)
    _, want = expected(x, False, 8, 64)
    for n in CACHE:
        got = torch.cat([pools[n][:2], pools[n][-2:]]).cpu().numpy()
        assert np.array_equal(got, want[n])
    outs = [torch.zeros((40, kv, dim), device="cuda") for _ in range(2)]
    S.seedlm_qcache_read(*cache, d["slots"], *outs)
    for got, name in zip(outs, "kv"):
        at = x["slots"] // size, x["slots"] % size
        ref, _ = Q.values(want[name + "_cache"][at], want[name + "_scale"][at], 8)
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= 2 * R.U32 * np.abs(ref))
    del pools, cache
    torch.cuda.empty_cache()


def test_another_stream_and_a_graph():
    import torch

    import prng_seeded_decode_amd as S

    x = make([10], 20, 4, 2, 128, 128, True, 16, 4, 4, 64)
    d = device(x, True)
    cache = [d[n] for n in CACHE]
    q_out, k_out, v_out = torch.zeros_like(d["q"]), torch.zeros_like(d["k"]), torch.zeros_like(d["v"])
    calls = [S.QCacheAppendCall(d["q"], d["k"], d["v"], d["cos"], d["sin"], d["positions"],
                                d["slots"], q_out, *cache),
             S.QCacheReadCall(*cache, d["slots"], k_out, v_out)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for call in calls:
            call()
    rng = np.random.default_rng(1)
    for step in range(4):
        x["slots"] = rng.permutation(64)[:20]
        x["v"] = rng.standard_normal(x["v"].shape).astype(np.float16)
        x.update({n: t.cpu().numpy() for n, t in zip(CACHE, cache)})
        _, want = expected(x, False, 4, 64)
        d["slots"].copy_(torch.from_numpy(x["slots"].astype(np.int32)))
        d["v"].copy_(torch.from_numpy(x["v"]))
        torch.cuda.synchronize()
        if step % 2:
            graph.replay()
        else:
            for call in calls:
                call(stream=side)
        torch.cuda.synchronize()
        for n, t in zip(CACHE, cache):
            assert np.array_equal(t.cpu().numpy(), want[n])
        at = x["slots"] // 16, x["slots"] % 16
        ref, _ = Q.values(want["v_cache"][at], want["v_scale"][at], 4)
        assert np.all(np.abs(v_out.double().cpu().numpy() - ref) <= R.rounding(ref, True) + R.U32 * np.abs(ref))


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("kv,dim,bits,groups", [(1, 64, 4, 2), (3, 64, 8, 1), (8, 128, 4, 4), (5, 128, 8, 1),
                                                (40, 128, 4, 1), (2, 256, 4, 1), (7, 256, 8, 4)])
def test_a_large_read_gives_what_small_ones_do(kv, dim, bits, groups, f16):
    # outputs of more than 32 MB go out another way than small ones
    import torch

    import prng_seeded_decode_amd as S

    tokens = (36 << 20) // (2 * kv * dim * (2 if f16 else 4)) + 3
    x = make([11, kv, dim], 1, 1, kv, dim, 0, True, 16, 50, bits, dim // groups)
    cache = [device({n: x[n] for n in CACHE}, True)[n] for n in CACHE]
    slots = np.random.default_rng(1).integers(-20, 820, tokens).astype(np.int32)
    slots = torch.from_numpy(slots).cuda()
    dt = torch.float16 if f16 else torch.float32
    both = torch.full((tokens, 2, kv, dim), 9.0, dtype=dt, device="cuda")
    S.seedlm_qcache_read(*cache, slots, both[:, 0], both[:, 1])
    part = 4001
    for at in range(0, tokens, part):
        n = min(part, tokens - at)
        k, v = (torch.full((n, kv, dim), 8.0, dtype=dt, device="cuda") for _ in range(2))
        S.seedlm_qcache_read(*cache, slots[at: at + n], k, v)
        assert torch.equal(both[at: at + n, 0], k) and torch.equal(both[at: at + n, 1], v), at
    one = torch.full((2 * tokens, kv, dim), 9.0, dtype=dt, device="cuda")
    S.seedlm_qcache_read(*cache, slots.repeat(2), None, one)
    assert torch.equal(one[:tokens], both[:, 1]) and torch.equal(one[tokens:], both[:, 1])


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("heads,kv,dim,rot,interleaved", [(40, 8, 128, 128, False), (9, 3, 256, 64, True),
                                                          (32, 32, 64, 64, True), (3, 1, 128, 32, False)])
def test_a_large_append_gives_what_small_ones_do(heads, kv, dim, rot, interleaved, f16):
    # q of more than 32 MB goes out another way than small ones
    import torch

    import prng_seeded_decode_amd as S

    tokens = (33 << 20) // (heads * dim * (2 if f16 else 4)) + 3
    size = 16
    x = make([12, heads, dim], 5, heads, kv, dim, rot, f16, size, tokens // size + 1, 4, dim // 2)
    g = torch.Generator(device="cuda").manual_seed(4)
    d = device(x, True)
    for k, h in (("q", heads), ("k", kv), ("v", kv)):
        d[k] = torch.randn((tokens, h, dim), generator=g, device="cuda").to(d[k].dtype)
    d["positions"] = torch.randint(-1, 98, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    d["slots"] = torch.randperm((tokens // size + 1) * size, generator=g, device="cuda")[:tokens].int()
    results = []
    for part in (tokens, 777):
        cache = [d[n].clone() for n in CACHE]
        q_out = torch.full_like(d["q"], 7.0)
        for at in range(0, tokens, part):
            e = {k: d[k][at: at + part] for k in ("q", "k", "v", "positions", "slots")}
            S.seedlm_qcache_append(e["q"], e["k"], e["v"], d["cos"], d["sin"], e["positions"],
                                   e["slots"], q_out[at: at + part], *cache, interleaved=interleaved)
        results.append([q_out, *cache[:2], *(t.view(torch.int16) for t in cache[2:])])
    for a, b in zip(*results):
        assert torch.equal(a, b)
