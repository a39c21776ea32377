"""seedlm_qcache_attend against softmax attention in 64 bits over what the cache stands for, element
by element within the bounds of qcache_ref.attend."""
import numpy as np
import pytest

import qcache_ref as Q

pytestmark = pytest.mark.gpu


def make(seed, lens, heads, kv, dim, size, f16, bits=4, groups=1, head_major=False, spread=1.5, pad=0):
    """Requests over shuffled pages.  Rows that no request owns - the rest of last pages, other
    pages - have NaN and infinite pairs, table entries past a request's pages are wild."""
    import torch

    rng = np.random.default_rng(seed)
    n = len(lens)
    held = [-(-v // size) for v in lens]
    pages = sum(held) + 3
    order = rng.permutation(pages)
    most = max(max(held), 1)
    table = rng.choice([-1, 2 ** 31 - 1, -2 ** 31, pages], (n, most))
    x = {"lens": np.array(lens), "table": table, "bits": bits}
    pools = {}
    for name, level in (("k", 6.0), ("v", 3.0)):
        codes = rng.integers(0, 256, (pages, size, kv, dim * bits // 8)).astype(np.uint8)
        pairs = np.full((pages, size, kv, groups, 2), np.nan, np.float16)
        pairs[::2] = np.inf
        pools[name] = codes, pairs
    rows = {b: [] for b in range(n)}
    at = 0
    for b, v in enumerate(lens):
        for t in range(v):
            table[b, t // size] = order[at + t // size]
            rows[b].append((table[b, t // size], t % size))
        at += held[b]
    for name, level in (("k", 6.0), ("v", 3.0)):
        codes, pairs = pools[name]
        for b in range(n):
            if not rows[b]:
                continue
            p, t = np.array(rows[b]).T
            s = rng.uniform(0.5, 1.5, (len(p), kv, groups)) * level / (2 ** bits - 1)
            o = -s * (2 ** bits - 1) / 2 + 0.2 * rng.standard_normal(s.shape)
            pairs[p, t] = np.stack([s, o], -1).astype(np.float16)
    q = (rng.standard_normal((n, heads, dim)) * spread).astype(np.float16 if f16 else np.float32)

    def pool(a, wide=0):
        t = torch.from_numpy(a).cuda()
        if head_major:
            t = t.transpose(1, 2).contiguous().transpose(1, 2)
        if wide:
            w = torch.zeros((*t.shape[:3], t.shape[3] + wide), dtype=t.dtype, device="cuda")
            w[..., :-wide] = t
            t = w[..., :-wide]
        return t

    x.update(q=q, where=rows, cache=[pool(pools["k"][0], pad), pool(pools["v"][0], pad),
                                     pool(pools["k"][1]), pool(pools["v"][1])])
    x.update(dq=torch.from_numpy(q).cuda(), dtable=torch.from_numpy(table.astype(np.int32)).cuda(),
             dlens=torch.from_numpy(np.array(lens, np.int32)).cuda())
    x["terms"] = [terms(x, b) for b in range(n)]
    return x


def terms(x, b):
    """k, its terms' magnitude, v and its, of a request's tokens as the cache holds them."""
    at = x["where"][b]
    if not at:
        return [np.zeros((0, 1, 1))] * 4
    p, t = np.array(at).T
    out = []
    for codes, pairs in ((x["cache"][0], x["cache"][2]), (x["cache"][1], x["cache"][3])):
        out += Q.values(codes[p, t].cpu().numpy(), pairs[p, t].cpu().numpy(), x["bits"])
    return out


def run(x, scale=None, **kw):
    import torch

    import prng_seeded_decode_amd as S

    out = kw.pop("out", None)
    if out is None:
        out = torch.full(x["dq"].shape, 9.0, dtype=x["dq"].dtype, device="cuda")
    S.seedlm_qcache_attend(x["dq"], *x["cache"], x["dtable"], x["dlens"], out, scale=scale, **kw)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


def check(x, got, scale=None, lens=None, rows=None, q=None):
    q = x["q"] if q is None else q
    f16, dim = q.dtype == np.float16, q.shape[2]
    scale = np.float32(dim ** -0.5 if scale is None else scale).astype(np.float64)
    lens = x["lens"] if lens is None else lens
    for i in range(len(lens)):
        b = i if rows is None else rows[i]
        n = lens[i]
        if not 0 <= b < len(x["terms"]):
            n, b = 0, 0
        ref, tol = Q.attend(q[i].astype(np.float64), *(a[:n] for a in x["terms"][b]), scale, f16)
        err = np.abs(got[i] - ref)
        if f16:  # numbers of 65520 and more round to fp16's infinity
            err[(np.abs(ref) + tol >= 65520) & (got[i] == np.copysign(np.inf, ref))] = 0
        assert np.all(err <= tol), (i, b, n, float((err - tol).max()), float(err.max()))


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300, 0, 511, 700]
SHAPES = [
    (8, 8, 64, 16, 1, False, 0), (8, 1, 64, 1, 2, False, 16), (12, 2, 64, 24, 1, True, 0),
    (4, 4, 128, 16, 1, False, 0), (16, 2, 128, 48, 2, True, 0), (6, 2, 128, 7, 4, False, 0),
    (20, 1, 128, 64, 2, False, 16), (40, 1, 64, 16, 2, True, 0),
    (4, 2, 256, 16, 4, False, 0), (8, 1, 256, 100, 1, True, 0), (1, 1, 256, 256, 2, False, 0)]


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("heads,kv,dim,size,groups,head_major,pad", SHAPES)
def test_attend_matches_64_bits_over_lengths(heads, kv, dim, size, groups, head_major, pad, bits, f16):
    x = make([heads, kv, dim, size, bits], LENS, heads, kv, dim, size, f16, bits, groups, head_major,
             pad=pad)
    check(x, run(x))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attend_of_short_requests(dim):
    lens = [0, 1, 5, 33, 100, 128, 64]
    x = make([dim], lens, 8, 2, dim, 16, True)
    check(x, run(x))                       # the table holds at most 128 tokens
    x = make([dim, 1], [100, 200, 0, 300], 8, 2, dim, 16, True, 8, 2)
    check(x, run(x, max_len=90), lens=[90, 90, 0, 90])


@pytest.mark.parametrize("lens", [[20000], [9000, 1, 0, 12345, 128], [4097] * 3])
@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("bits,groups,dim", [(4, 1, 128), (4, 2, 64), (8, 4, 128), (4, 4, 256)])
def test_attend_over_long_caches(lens, f16, bits, groups, dim):
    x = make([len(lens), lens[0]], lens, 4, 2, dim, 16, f16, bits, groups, True)
    check(x, run(x))


@pytest.mark.parametrize("n", [257, 1000, 4096])
@pytest.mark.parametrize("f16", [True, False])
def test_attend_of_many_requests(n, f16):
    rng = np.random.default_rng(n)
    lens = [int(v) for v in rng.integers(0, 40, n)]
    lens[n // 2], lens[3], lens[n - 1] = 1500, 0, 300
    x = make([n], lens, 2, 1, 64, 16, f16)
    check(x, run(x))


def test_attend_limits_lengths_to_max_len_and_the_table():
    import torch

    x = make([3], [304, 40, 208], 4, 2, 128, 16, True)
    check(x, run(x, max_len=170), lens=[170, 40, 170])
    # past any table, negative, and past the request's own pages (whose entries are no pages)
    x["dlens"] = torch.tensor([10 ** 9, -3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    check(x, run(x), lens=[304, 0, 208])


@pytest.mark.parametrize("lens", [[100, 64, 50], [2000, 640, 50]])
def test_attend_skips_pages_outside_the_cache(lens):
    import torch

    x = make([4, lens[0]], lens, 4, 2, 128, 16, True, 4, 2)
    table = x["table"].copy()
    table[0, 2], table[1, :] = -1, 10 ** 6
    x["dtable"] = torch.from_numpy(table.astype(np.int32)).cuda()
    keep = np.r_[0:32, 48:lens[0]]
    x["terms"][0] = [a[keep] for a in x["terms"][0]]
    got = run(x)
    check(x, got, lens=[lens[0] - 16, 0, 50])
    assert (got[1] == 0).all()


@pytest.mark.parametrize("f16", [True, False])
def test_attend_with_extreme_scores(f16):
    for scale in (0.0, 5.0, -3.0, 1e-6):
        x = make([6], [700, 129, 1], 4, 2, 128, 16, f16, 4, 2)
        check(x, run(x, scale=scale), scale=scale)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("bits", [4, 8])
def test_one_heavy_token_beside_many_light_ones(f16, bits):
    # 20000 tokens of one score beside one that is e^12 times as heavy
    import torch

    x = make([9], [20000], 1, 1, 64, 16, f16, bits, 1, spread=0.0)
    ks = x["cache"][2]
    p, t = np.array(x["where"][0]).T
    ks[p, t] = 0.0
    ks[p[777], t[777], 0, 0] = torch.tensor([0.0, 12.0 / 64], dtype=torch.float16)
    x["q"][:] = 1.0
    x["dq"] = torch.from_numpy(x["q"]).cuda()
    x["terms"][0] = terms(x, 0)
    check(x, run(x, scale=1.0), scale=1.0)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dim,bits,groups", [(128, 4, 1), (64, 8, 2), (256, 4, 4)])
def test_scales_of_values_over_fp16s_whole_range(f16, dim, bits, groups):
    # scales that grow, shrink and vanish from token to token: each tile has another largest one
    import torch

    rng = np.random.default_rng(5)
    lens = [1500, 200, 40]
    for power in (rng.integers(-24, 13, 1500), np.sort(rng.integers(-24, 13, 1500)),
                  np.sort(rng.integers(-24, 13, 1500))[::-1], np.full(1500, -24), np.full(1500, 12)):
        x = make([15, dim], lens, 4, 2, dim, 16, f16, bits, groups)
        for b in range(3):
            p, t = np.array(x["where"][b]).T
            s = torch.from_numpy(2.0 ** power[: lens[b]].astype(np.float64)).half().cuda()
            x["cache"][3][p, t, :, :, 0] = s[:, None, None]
            x["terms"][b] = terms(x, b)
        check(x, run(x))


def test_small_and_large_queries():
    import torch

    for f16, powers in ((False, (-60, -30, 0, 30)), (True, (-14, -8, 0, 10))):
        x = make([10], [300, 200, 77], 4, 2, 64, 16, f16)
        for power in powers:
            q = (x["q"].astype(np.float32) * np.float32(2.0) ** power).astype(x["q"].dtype)
            scale = 0.125 * 2.0 ** -power
            check(x, run(dict(x, dq=torch.from_numpy(q).cuda()), scale=scale), scale=scale, q=q)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("lens", [[200, 150, 90], [2000, 1500, 90, 0, 1300]])
@pytest.mark.parametrize("dim,bits,groups", [(64, 4, 2), (128, 8, 1), (256, 4, 2)])
def test_nan_keeps_to_its_own_request_head_and_group(dim, bits, groups, lens, f16):
    x = make([41, dim], lens, 4, 2, dim, 16, f16, bits, groups)
    clean = run(x)
    check(x, clean)
    page, row = x["where"][1][53]
    part = slice(0, dim // groups)
    x["cache"][3][page, row, 0, 0, 0] = float("nan")
    got = run(x)
    assert np.isnan(got[1, :2, part]).all()
    got[1, :2, part] = clean[1, :2, part]
    assert np.array_equal(got, clean)
    x["cache"][2][page, row, 1, groups - 1, 1] = float("inf")
    got = run(x)
    assert np.isnan(got[1, 2:]).all()
    got[1] = clean[1]
    assert np.array_equal(got, clean)


def test_attend_in_place_strided_rows_another_stream_and_a_graph():
    import torch

    import prng_seeded_decode_amd as S

    x = make([12], [200, 1500, 0, 33], 8, 2, 128, 16, True, 4, 2)
    plain = run(x)
    n = len(x["lens"])
    wide = torch.zeros((n, 8 * 128 + 64), dtype=torch.float16, device="cuda")
    rows = wide[:, : 8 * 128].view(n, 8, 128)
    rows.copy_(x["dq"])
    assert np.array_equal(run(dict(x, dq=rows), out=rows), plain)
    assert (wide[:, 8 * 128:] == 0).all()
    wide_table = torch.full((n, x["dtable"].shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide_table[:, 2:-3] = x["dtable"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert np.array_equal(run(dict(x, dtable=wide_table[:, 2:-3]), stream=side), plain)
    out = torch.zeros_like(x["dq"])
    call = S.QCacheAttendCall(x["dq"], *x["cache"], x["dtable"], x["dlens"], out)
    with torch.cuda.stream(side):
        call()  # the stream's scratch exists before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for lens in ([200, 1500, 0, 33], [7, 1000, 0, 32], [0, 0, 0, 1], [200, 129, 0, 33]):
        x["dlens"].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        check(x, got, lens=lens)
        assert np.array_equal(got, run(x))


def test_attend_reaches_past_32_bit_offsets():
    # code pools past 2^32 bytes; only the pages in use are ever written or read
    import torch

    size, kv, dim = 16, 8, 256
    pages = 2 ** 32 // (size * kv * dim) + 9
    x = make([13], [1300, 70, 0], 8, kv, dim, size, True, 8, 1)
    where = {}
    for b in range(3):
        for j in range(-(-int(x["lens"][b]) // size)):
            where[b, j] = pages - 1 - j if (b + j) % 2 == 0 else j + 200 * b
    assert len(set(where.values())) == len(where)
    pools = []
    for a in x["cache"]:
        pool = torch.empty((pages, *a.shape[1:]), dtype=a.dtype, device="cuda")
        for (b, j), at in where.items():
            pool[at] = a[int(x["table"][b, j])]
        pools.append(pool)
    table = np.full_like(x["table"], -1)
    for (b, j), at in where.items():
        table[b, j] = at
    check(x, run(dict(x, cache=pools, dtable=torch.from_numpy(table.astype(np.int32)).cuda())))
    del pools
    torch.cuda.empty_cache()


def run_rows(x, q, rows, lens, **kw):
    import torch

    import prng_seeded_decode_amd as S

    i32 = lambda a: torch.tensor([int(v) for v in a], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    S.seedlm_qcache_attend(q, *x["cache"], x["dtable"], i32(lens), out, rows=i32(rows), **kw)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("heads,kv,dim,bits,groups", [
    (8, 2, 128, 4, 1), (4, 4, 64, 8, 2), (6, 2, 128, 4, 4), (6, 1, 256, 4, 2), (20, 1, 64, 4, 1),
    (5, 1, 64, 4, 1), (16, 1, 128, 8, 1)])
def test_several_queries_per_request(heads, kv, dim, bits, groups, f16):
    # any order of rows, several of one request at different lengths, rows outside the table
    import torch

    x = make([14, heads], [300, 70, 1000], heads, kv, dim, 16, f16, bits, groups)
    g = torch.Generator(device="cuda").manual_seed(7)
    rows = [2, 0, 0, -1, 1, 2, 3, 0, 2 ** 31 - 1, 1, 1, 1, 1, 2, 2]
    lens = [1000, 300, 17, 50, 70, 513, 20, 0, 1, 1, 0, 70, 3, 1000, 1]
    q = torch.randn((len(rows), heads, dim), generator=g, device="cuda").to(x["dq"].dtype)
    host = q.cpu().numpy()
    check(x, run_rows(x, q, rows, lens), lens=lens, rows=rows, q=host)
    check(x, run_rows(x, q, rows, lens, max_len=250), lens=np.minimum(lens, 250), rows=rows, q=host)
    short = np.minimum(lens, 60)
    check(x, run_rows(x, q, rows, short, max_len=60), lens=short, rows=rows, q=host)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("heads,kv,dim,bits", [(8, 2, 128, 4), (4, 4, 64, 8), (6, 1, 256, 4)])
def test_hundreds_of_queries_of_a_few_requests(heads, kv, dim, bits, f16):
    # pieces of prompts behind cached tokens, single tokens, padding rows; in a plan's order,
    # and in any other
    import torch

    ends, fresh = [150, 41, 700, 7, 1100, 0], [150, 1, 80, 7, 40, 0]
    x = make([44, dim], ends, heads, kv, dim, 16, f16, bits, 1, True)
    rows = np.array([b for b in range(6) for _ in range(fresh[b])] + [-1] * 5)
    lens = np.array([ends[b] - fresh[b] + i + 1 for b in range(6) for i in range(fresh[b])] + [0] * 5)
    g = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randn((len(rows), heads, dim), generator=g, device="cuda").to(x["dq"].dtype)
    for perm in (np.arange(len(rows)), np.random.default_rng(3).permutation(len(rows))):
        at = torch.from_numpy(perm).cuda()
        got = run_rows(x, q[at], rows[perm], lens[perm])
        check(x, got, lens=lens[perm], rows=rows[perm], q=q[at].cpu().numpy())


def test_nan_past_one_querys_length_but_not_anothers():
    # queries that share their reading: what only the longer one attends to reaches it alone
    import torch

    for heads, kv in ((4, 2), (16, 2)):
        x = make([16, heads], [400], heads, kv, 128, 16, True, 4, 2)
        q = torch.randn((6, heads, 128), device="cuda").half()
        lens, rows = [100, 400, 390, 380, 10, 381], [0] * 6
        clean = run_rows(x, q, rows, lens)
        check(x, clean, lens=lens, rows=rows, q=q.cpu().numpy())
        page, row = x["where"][0][380]
        x["cache"][3][page, row, :, :, :] = float("nan")
        x["cache"][2][page, row, :, :, 0] = float("inf")
        got = run_rows(x, q, rows, lens)
        bad = np.array([False, True, True, False, False, True])
        assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], clean[~bad])


def test_attend_with_a_table_that_holds_more_than_32_bits_of_tokens():
    # 2^21 pages of 2048 tokens: refused by its own bound, taken with the caller's
    import torch

    import prng_seeded_decode_amd as S

    x = make([15], [90], 4, 2, 64, 2048, True)
    wide = torch.full((1, 2 ** 21), -1, dtype=torch.int32, device="cuda")
    wide[:, 0] = x["dtable"][:, 0]
    y = dict(x, dtable=wide)
    with pytest.raises(S.SeedLMError) as refused:
        run(y)
    assert refused.value.status == S.E_UNSUPPORTED
    with pytest.raises(ValueError):
        run(y, max_len=-1)
    check(x, run(y, max_len=100))


def widen(x, most, wild=-1):
    """The same requests in a table of `most` pages a row."""
    import torch

    table = torch.full((x["table"].shape[0], most), wild, dtype=torch.int32, device="cuda")
    table[:, : x["table"].shape[1]] = x["dtable"]
    return dict(x, dtable=table)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("heads,kv,dim,size,groups,head_major", [
    (8, 2, 128, 16, 1, False), (20, 1, 128, 48, 2, True), (4, 4, 128, 7, 4, False),
    (4, 2, 256, 16, 2, True), (18, 1, 256, 100, 4, False)])
def test_codes_past_the_caches(heads, kv, dim, size, groups, head_major, bits, f16):
    # calls that may read more than 256 MB
    lens = [0, 1, 33, 128, 129, 700, 3000, 255, 2049, 0]
    row = dim * bits // 8 + 4 * groups
    most = 2 ** 28 // (len(lens) * kv * 2 * row * size) + 2
    x = widen(make([heads, dim, size, 7], lens, heads, kv, dim, size, f16, bits, groups, head_major), most,
              wild=2 ** 31 - 1)
    check(x, run(x))


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 200])
@pytest.mark.parametrize("dim,groups", [(128, 1), (64, 2), (256, 1)])
def test_split_of_any_number_of_requests(n, dim, groups):
    # up to 64 queries are counted in registers, more in LDS; a wide table has them split
    rng = np.random.default_rng([n, dim])
    lens = [int(v) for v in np.exp(rng.uniform(0, np.log(900), n)).astype(int) * rng.integers(0, 2, n)]
    lens[n // 2] = 1300
    x = widen(make([n, dim], lens, 4, 2, dim, 16, True, 4, groups), 400)
    check(x, run(x))


@pytest.mark.parametrize("heads,kv", [(32, 2), (7, 7), (24, 8), (3, 1)])
def test_rows_that_repeat_with_and_without_a_split(heads, kv):
    # blocks of queries whose rows change inside, repeat after others, and end in padding
    import torch

    x = make([17, heads], [900, 40, 333], heads, kv, 64, 16, True, 4, 1)
    rows = np.array([0] * 17 + [1] + [0] * 3 + [2] * 30 + [-1] * 4 + [1] * 9 + [2])
    rng = np.random.default_rng(1)
    lens = np.array([int(rng.integers(0, len(x["where"][r]))) if r >= 0 else 5 for r in rows])
    q = torch.randn((len(rows), heads, 64), device="cuda").half()
    host = q.cpu().numpy()
    want = run_rows(x, q, rows, lens)
    check(x, want, lens=lens, rows=rows, q=host)
    got = run_rows(widen(x, 9000), q, rows, lens)
    check(x, got, lens=lens, rows=rows, q=host)
    # NaN behind every length of a row reaches none of its queries
    page, row = x["where"][2][332]
    x["cache"][3][page, row] = float("nan")
    assert np.array_equal(run_rows(x, q, rows, lens), want)
    assert np.array_equal(run_rows(widen(x, 9000), q, rows, lens), got)


@pytest.mark.parametrize("bits,groups,dim", [(4, 1, 64), (4, 4, 128), (4, 2, 256), (8, 1, 64), (8, 2, 128)])
def test_sums_of_fp32_calls_keep_their_low_bits(bits, groups, dim):
    # The bounds element by element are of the worst case; errors on one side hide below them.
    # So the root mean square over all outputs, relative to the terms' magnitudes: a weight is
    # cut to 22 bits in two parts (2^-21), sums and products round 8 times at their size, and a
    # score errs by 8 roundings of its terms' magnitudes, independently from token to token, so
    # that 1 / sqrt(tokens that count) of it is left.
    n = 1024
    x = make([bits, groups, dim, 77], [n], 8, 8, dim, 64, False, bits, groups)
    got = run(x)[0]
    q = x["q"][0].astype(np.float64)
    k, kmag, v, vmag = x["terms"][0]
    scale = np.float64(np.float32(dim ** -0.5))
    err, terms_, left = [], [], []
    for h in range(8):
        s = k[:, h] @ q[h] * scale
        w = np.exp(s - s.max())
        w /= w.sum()
        err.append(got[h] - w @ v[:, h])
        terms_.append(w @ vmag[:, h])
        left.append((kmag[:, h] @ np.abs(q[h])).max() * scale * np.sqrt((w ** 2).sum()))
    size = np.sqrt(np.mean(np.square(terms_)))
    bound = 2.0 ** -21 + 8 * Q.U32 + 8 * Q.U32 * max(left)
    assert np.sqrt(np.mean(np.square(err))) <= bound * size


@pytest.mark.parametrize("shared", [False, True])
def test_the_most_queries_of_the_widest_heads_in_the_split_form(shared):
    # the largest LDS of any call: the entries and sums of 4096 queries beside partials of 256
    import torch

    n = 4096
    lens = np.random.default_rng(5).integers(0, 3, n)
    lens[[7, 2000, 4095]] = 2300, 1, 1100
    x = make([256, n, shared], list(lens), 2, 1, 256, 32, True, 4, 2)
    rows = torch.arange(n, dtype=torch.int32, device="cuda") if shared else None
    check(x, run(x, rows=rows))
