"""seedlm_cache_attend against softmax attention in 64 bits, element by element within the
bounds of serve_ref.attend."""
import numpy as np
import pytest

import serve_ref as R

pytestmark = pytest.mark.gpu


def make(seed, lens, heads, kv, dim, size, f16, head_major=False, spread=1.5, junk=True, pad=0):
    """Requests over shuffled pages.  Everything that no request owns - the rest of last pages,
    other pages - holds NaN and infinities, table entries past a request's pages are wild."""
    import torch

    rng = np.random.default_rng(seed)
    n = len(lens)
    held = [-(-v // size) for v in lens]
    pages = sum(held) + 3
    order = rng.permutation(pages)
    most = max(max(held), 1)
    table = rng.choice([-1, 2 ** 31 - 1, -2 ** 31, pages], (n, most))
    keys, values = [], []
    shape = (pages, size, kv, dim)
    kc = np.full(shape, np.nan if junk else 0.0, np.float16)
    vc = np.full(shape, np.inf if junk else 0.0, np.float16)
    at = 0
    for b, v in enumerate(lens):
        k = rng.standard_normal((v, kv, dim)).astype(np.float16)
        w = rng.standard_normal((v, kv, dim)).astype(np.float16)
        keys.append(k.astype(np.float64))
        values.append(w.astype(np.float64))
        for j in range(held[b]):
            page = order[at + j]
            table[b, j] = page
            part = slice(j * size, min((j + 1) * size, v))
            kc[page, : part.stop - part.start] = k[part]
            vc[page, : part.stop - part.start] = w[part]
        at += held[b]
    q = (rng.standard_normal((n, heads, dim)) * spread).astype(np.float16 if f16 else np.float32)

    def cache(a):
        t = torch.from_numpy(a).cuda()
        if head_major:
            t = t.transpose(1, 2).contiguous().transpose(1, 2)
        if pad:
            wide = torch.zeros((pages, size, kv, dim + pad), dtype=t.dtype, device="cuda")
            wide[..., :dim] = t
            t = wide[..., :dim]
        return t

    return {"q": q, "keys": keys, "values": values, "lens": np.array(lens), "table": table,
            "k_cache": cache(kc), "v_cache": cache(vc),
            "dq": torch.from_numpy(q).cuda(),
            "dtable": torch.from_numpy(table.astype(np.int32)).cuda(),
            "dlens": torch.from_numpy(np.array(lens, np.int32)).cuda()}


def run(x, scale=None, **kw):
    import torch

    import prng_seeded_decode_amd as S

    out = kw.pop("out", None)
    if out is None:
        out = torch.full(x["q"].shape, 9.0, dtype=x["dq"].dtype, device="cuda")
    S.seedlm_cache_attend(x["dq"], x["k_cache"], x["v_cache"], x["dtable"], x["dlens"], out,
                          scale=scale, **kw)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


def check(x, got, scale=None, lens=None):
    f16 = x["q"].dtype == np.float16
    dim = x["q"].shape[2]
    scale = np.float32(dim ** -0.5 if scale is None else scale).astype(np.float64)
    for b in range(len(x["lens"])):
        n = x["lens"][b] if lens is None else lens[b]
        ref, tol = R.attend(x["q"][b].astype(np.float64), x["keys"][b][:n], x["values"][b][:n],
                            scale, f16)
        err = np.abs(got[b] - ref)
        assert np.all(err <= tol), (b, n, float((err - tol).max()), float(err.max()))


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300, 0, 511, 700]


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("heads,kv,dim,size,head_major,pad", [
    (8, 8, 64, 16, False, 0), (8, 1, 64, 1, False, 8), (12, 2, 64, 24, True, 0),
    (4, 4, 128, 16, False, 0), (16, 2, 128, 48, True, 0), (6, 2, 128, 7, False, 0),
    (20, 1, 128, 64, False, 16), (40, 1, 64, 16, True, 0),
    (4, 2, 256, 16, False, 0), (8, 1, 256, 100, True, 0), (1, 1, 256, 256, False, 0),
])
def test_attend_matches_64_bits_over_lengths(heads, kv, dim, size, head_major, pad, f16):
    x = make([heads, kv, dim, size], LENS, heads, kv, dim, size, f16, head_major, pad=pad)
    check(x, run(x))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attend_where_no_request_needs_a_split(dim):
    lens = [0, 1, 5, 33, 100, 128, 64]
    x = make([dim], lens, 8, 2, dim, 16, True)
    check(x, run(x))                       # the table holds at most 128 tokens
    x = make([dim, 1], [100, 200, 0, 300], 8, 2, dim, 16, True)
    check(x, run(x, max_len=90), lens=[90, 90, 0, 90])


@pytest.mark.parametrize("lens", [[20000], [9000, 1, 0, 12345, 128], [4097] * 3])
@pytest.mark.parametrize("f16", [True, False])
def test_attend_over_long_caches(lens, f16):
    x = make([len(lens), lens[0]], lens, 4, 2, 128, 16, f16)
    check(x, run(x))


@pytest.mark.parametrize("n", [257, 1000, 4096])
def test_attend_of_many_requests(n):
    rng = np.random.default_rng(n)
    lens = [int(v) for v in rng.integers(0, 40, n)]
    lens[n // 2] = 900
    x = make([n], lens, 2, 1, 64, 16, True)
    check(x, run(x))


def test_attend_limits_lengths_to_max_len_and_the_table():
    import torch

    x = make([3], [304, 40, 208], 4, 2, 128, 16, True)
    check(x, run(x, max_len=170), lens=[170, 40, 170])
    # past any table, negative, and past the request's own pages (whose entries are no pages)
    x["dlens"] = torch.tensor([10 ** 9, -3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    check(x, run(x), lens=[304, 0, 208])


def test_attend_skips_pages_outside_the_cache():
    import torch

    x = make([4], [100, 64, 50], 4, 2, 128, 16, True)
    table = x["table"].copy()
    table[0, 2], table[1, :] = -1, 10 ** 6
    x["dtable"] = torch.from_numpy(table.astype(np.int32)).cuda()
    keep = np.r_[0:32, 48:100]
    x["keys"][0], x["values"][0] = x["keys"][0][keep], x["values"][0][keep]
    got = run(x)
    check(x, got, lens=[84, 0, 50])
    assert (got[1] == 0).all()


@pytest.mark.parametrize("f16", [True, False])
def test_attend_with_extreme_scores(f16):
    lens = [700, 129, 1]
    for scale in (0.0, 5.0, -3.0, 1e-6):
        x = make([6], lens, 4, 2, 128, 16, f16)
        check(x, run(x, scale=scale), scale=scale)
    # many tokens of equal weight beside one that is e^12 times as heavy
    x = make([8], [20000], 1, 1, 64, 16, f16, spread=0.0)
    got = run(x)
    assert np.all(np.abs(got[0, 0] - x["values"][0][:, 0].mean(0)) <= 2.0 ** -10)
    x = make([9], [20000], 1, 1, 64, 16, f16, spread=0.0)
    x["q"][0, 0, 0] = 1.0
    x["k_cache"][:, :, :, 0] = 0.0
    x["keys"][0][:, :, 0] = 0.0
    x["keys"][0][777, 0, 0] = 12.0
    x["k_cache"][int(x["table"][0, 777 // 16]), 777 % 16, 0, 0] = 12.0
    import torch

    x["dq"] = torch.from_numpy(x["q"]).cuda()
    check(x, run(x, scale=1.0), scale=1.0)


def test_attend_keeps_small_fp32_queries():
    # rows whose elements lie far below fp16's range, or far above it
    x = make([10], [300, 200, 77], 4, 2, 64, 16, False)
    for power in (-60, -30, 0, 30):
        q = (x["q"] * np.float32(2.0) ** power).astype(np.float32)
        import torch

        y = dict(x, q=q, dq=torch.from_numpy(q).cuda())
        scale = 0.125 * 2.0 ** -power
        check(y, run(y, scale=scale), scale=scale)


def test_attend_keeps_nan_to_its_own_request_and_head():
    x = make([11], [200, 150, 90], 4, 2, 128, 16, True)
    clean = run(x)
    page, row = int(x["table"][1, 3]), 5
    x["k_cache"][page, row, 1, 7] = float("nan")
    got = run(x)
    assert np.isnan(got[1, 2:]).all()
    got[1, 2:] = clean[1, 2:]
    assert np.array_equal(got, clean)


def test_attend_in_place_strided_rows_another_stream_and_a_graph():
    import torch

    import prng_seeded_decode_amd as S

    x = make([12], [200, 1500, 0, 33], 8, 2, 128, 16, True)
    plain = run(x)
    n = len(x["lens"])
    wide = torch.zeros((n, 8 * 128 + 64), dtype=torch.float16, device="cuda")
    rows = wide[:, : 8 * 128].view(n, 8, 128)
    rows.copy_(x["dq"])
    y = dict(x, dq=rows)
    assert np.array_equal(run(y, out=rows), plain)
    assert (wide[:, 8 * 128:] == 0).all()
    wide_table = torch.full((n, x["dtable"].shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide_table[:, 2:-3] = x["dtable"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert np.array_equal(run(dict(x, dtable=wide_table[:, 2:-3]), stream=side), plain)
    out = torch.zeros_like(x["dq"])
    call = S.CacheAttendCall(x["dq"], x["k_cache"], x["v_cache"], x["dtable"], x["dlens"], out)
    with torch.cuda.stream(side):
        call()  # the stream's scratch exists before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for lens in ([200, 1500, 0, 33], [7, 1000, 0, 32], [0, 0, 0, 1], [200, 129, 0, 33]):
        x["dlens"].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        check(x, got, lens=lens)
        assert np.array_equal(got, run(x))


def test_attend_reaches_past_32_bit_offsets():
    # pools of 2^32 elements and more; only the pages in use are ever written or read
    import torch

    size, kv, dim = 16, 8, 128
    pages = 2 ** 32 // (size * kv * dim) + 9
    x = make([13], [40, 70], 8, kv, dim, size, True)
    pools = []
    where = {}
    for name in ("k_cache", "v_cache"):
        pool = torch.empty((pages, size, kv, dim), dtype=torch.float16, device="cuda")
        for b in range(2):
            for j in range(-(-int(x["lens"][b]) // size)):
                at = where.setdefault((b, j), pages - 1 - 3 * b - j if b else j)
                pool[at] = x[name][int(x["table"][b, j])]
        pools.append(pool)
    table = np.full_like(x["table"], -1)
    for (b, j), at in where.items():
        table[b, j] = at
    y = dict(x, k_cache=pools[0], v_cache=pools[1],
             dtable=torch.from_numpy(table.astype(np.int32)).cuda())
    check(x, run(y))
    del pools, y
    torch.cuda.empty_cache()


def test_attend_of_several_queries_per_request():
    # queries in any order of rows, several of one request at different lengths, rows outside
    # the table: each equals the same query attending alone
    import torch

    import prng_seeded_decode_amd as S

    x = make([14], [300, 70, 1000], 8, 2, 128, 16, True)
    rows = [2, 0, 0, -1, 1, 2, 3, 0, 2 ** 31 - 1, 1]
    lens = [1000, 300, 17, 50, 70, 513, 20, 0, 1, 1]
    q = torch.randn((len(rows), 8, 128), device="cuda").half()
    out = torch.full_like(q, 3.0)
    S.seedlm_cache_attend(q, x["k_cache"], x["v_cache"], x["dtable"],
                          torch.tensor(lens, dtype=torch.int32, device="cuda"), out,
                          rows=torch.tensor(rows, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    for i, (row, n) in enumerate(zip(rows, lens)):
        if not 0 <= row < 3:
            n, row = 0, 0
        ref, tol = R.attend(q[i].double().cpu().numpy(), x["keys"][row][:n], x["values"][row][:n],
                            np.float64(np.float32(128 ** -0.5)), True)
        assert np.all(np.abs(got[i] - ref) <= tol), i


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
