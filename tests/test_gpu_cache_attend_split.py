"""seedlm_cache_attend where work is split over the lengths and where keys and values pass the
caches, element by element within the bounds of serve_ref.attend.

The host sees only the table's width, so a wide table selects either form at short lengths."""
import numpy as np
import pytest

import serve_ref as R
from test_gpu_cache_attend import check, make

pytestmark = pytest.mark.gpu

STREAMED = 2 ** 28  # bytes that a call may read: more of them pass the caches


def widen(x, most, wild=-1):
    """The same requests in a table of `most` pages a row."""
    import torch

    table = torch.full((x["table"].shape[0], most), wild, dtype=torch.int32, device="cuda")
    table[:, : x["table"].shape[1]] = x["dtable"]
    return dict(x, dtable=table)


def run_split(x, scale=None, **kw):
    import torch

    import prng_seeded_decode_amd as S

    out = torch.full(x["q"].shape, 9.0, dtype=x["dq"].dtype, device="cuda")
    call = S.CacheAttendCall(x["dq"], x["k_cache"], x["v_cache"], x["dtable"], x["dlens"], out,
                             scale=scale, **kw)
    assert call.scratch_bytes() > 0
    call()
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


LENS = [0, 1, 2, 31, 32, 33, 127, 128, 129, 0, 700, 3000, 255, 1, 1025, 16, 2049, 0]


@pytest.mark.parametrize("n", [257, 1000, 4096])
@pytest.mark.parametrize("f16", [True, False])
def test_many_requests(n, f16):
    rng = np.random.default_rng(n)
    lens = [int(v) for v in rng.integers(0, 40, n)]
    lens[n // 2], lens[3], lens[n - 1] = 1500, 0, 300
    x = make([n, 1], lens, 4, 2, 64, 16, f16)
    check(x, run_split(x))


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("heads,kv,size,head_major", [
    (8, 8, 16, False), (12, 3, 24, True), (8, 1, 1, False), (40, 2, 64, True)])
def test_64_dimensions(heads, kv, size, head_major, f16):
    x = make([heads, kv, size], LENS, heads, kv, 64, size, f16, head_major)
    check(x, run_split(x))


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("heads,kv,dim,size,head_major,pad", [
    (8, 2, 128, 16, False, 0), (20, 1, 128, 48, True, 0), (4, 4, 128, 7, False, 8),
    (4, 2, 256, 16, False, 0), (18, 1, 256, 100, True, 0)])
def test_keys_and_values_past_the_caches(heads, kv, dim, size, head_major, pad, f16):
    most = STREAMED // (len(LENS) * kv * dim * 4 * size) + 2
    x = widen(make([heads, dim, size, 7], LENS, heads, kv, dim, size, f16, head_major, pad=pad), most,
              wild=2 ** 31 - 1)
    assert len(LENS) * most * size * kv * dim * 4 > STREAMED
    check(x, run_split(x))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("wide", [False, True])
def test_nan_stays_with_its_own_request_and_head(dim, wide):
    x = make([41, dim], [2000, 1500, 90, 0, 1300], 4, 2, dim, 16, True)
    if wide:
        x = widen(x, STREAMED // (5 * 2 * dim * 4 * 16) + 2)
    clean = run_split(x)
    check(x, clean)
    page = int(x["table"][1, 3])
    x["k_cache"][page, 5, 1, 7] = float("nan")
    got = run_split(x)
    assert np.isnan(got[1, 2:]).all()
    got[1, 2:] = clean[1, 2:]
    assert np.array_equal(got, clean)
    x["v_cache"][page, 6, 0, 9] = float("nan")
    got = run_split(x)
    assert np.isnan(got[1, :2, 9]).all() and np.isnan(got[1, 2:]).all()
    got[1] = clean[1]
    assert np.array_equal(got, clean)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_an_infinite_value_stays_with_its_own_dimension(dim, f16):
    x = make([45, dim], [2000, 1500, 90], 4, 2, dim, 16, f16)
    clean = run_split(x)
    x["v_cache"][int(x["table"][1, 3]), 6, 0, 9] = float("-inf")
    got = run_split(x)
    assert not np.isfinite(got[1, :2, 9]).any()
    got[1, :2, 9] = clean[1, :2, 9]
    assert np.array_equal(got, clean)


@pytest.mark.parametrize("f16", [True, False])
def test_pages_outside_the_cache_and_lengths_past_the_table(f16):
    import torch

    x = make([42], [2000, 640, 50], 4, 2, 128, 16, f16)
    table = x["table"].copy()
    table[0, 20], table[1, :] = -1, 10 ** 6
    x["dtable"] = torch.from_numpy(table.astype(np.int32)).cuda()
    x["dlens"] = torch.tensor([2 ** 31 - 1, 640, 50], dtype=torch.int32, device="cuda")
    keep = np.r_[0:320, 336:2000]
    x["keys"][0], x["values"][0] = x["keys"][0][keep], x["values"][0][keep]
    got = run_split(x)
    check(x, got, lens=[1984, 0, 50])
    assert (got[1] == 0).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("wide", [False, True])
def test_offsets_past_32_bits(dim, wide):
    # pools of 2^32 elements and more; only the pages in use are ever written or read
    import torch

    size, kv = 16, 8
    pages = 2 ** 32 // (size * kv * dim) + 9
    x = make([43, dim], [1300, 70, 0], 8, kv, dim, size, True)
    pools, where = [], {}
    for name in ("k_cache", "v_cache"):
        pool = torch.empty((pages, size, kv, dim), dtype=torch.float16, device="cuda")
        for b in range(3):
            for j in range(-(-int(x["lens"][b]) // size)):
                at = where.setdefault((b, j), pages - 1 - j if (b + j) % 2 == 0 else j + 200 * b)
                pool[at] = x[name][int(x["table"][b, j])]
        pools.append(pool)
    assert len(set(where.values())) == len(where)
    table = np.full_like(x["table"], -1)
    for (b, j), at in where.items():
        table[b, j] = at
    y = dict(x, k_cache=pools[0], v_cache=pools[1],
             dtable=torch.from_numpy(table.astype(np.int32)).cuda())
    if wide:
        y = widen(y, STREAMED // (3 * kv * dim * 4 * size) + 2)
    check(y, run_split(y))
    del pools, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (4, 4, 64), (6, 1, 256)])
def test_hundreds_of_queries_of_a_few_requests(heads, kv, dim, f16):
    # pieces of prompts behind cached tokens, single tokens, padding rows; in a plan's order,
    # and in any other
    import torch

    import prng_seeded_decode_amd as S

    ends, fresh = [150, 41, 700, 7, 1100, 0], [150, 1, 80, 7, 40, 0]
    x = make([44, dim], ends, heads, kv, dim, 16, f16)
    rows = [b for b in range(6) for _ in range(fresh[b])] + [-1] * 5
    lens = [ends[b] - fresh[b] + i + 1 for b in range(6) for i in range(fresh[b])] + [0] * 5
    n = len(rows)
    g = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randn((n, heads, dim), generator=g, device="cuda").to(x["dq"].dtype)
    host = q.double().cpu().numpy()
    scale = np.float64(np.float32(dim ** -0.5))
    refs = []
    for i in range(n):
        length, row = (lens[i], rows[i]) if rows[i] >= 0 else (0, 0)
        refs.append(R.attend(host[i], x["keys"][row][:length], x["values"][row][:length], scale, f16))
    for perm in (np.arange(n), np.random.default_rng(3).permutation(n)):
        out = torch.full_like(q, 3.0)
        i32 = lambda a: torch.from_numpy(np.asarray(a)[perm].astype(np.int32)).cuda()
        call = S.CacheAttendCall(q[torch.from_numpy(perm).cuda()], x["k_cache"], x["v_cache"],
                                 x["dtable"], i32(lens), out, rows=i32(rows))
        assert call.scratch_bytes() > 0
        call()
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        for at, i in enumerate(perm):
            ref, tol = refs[i]
            assert np.all(np.abs(got[at] - ref) <= tol), (i, rows[i], lens[i])
