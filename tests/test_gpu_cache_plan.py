"""seedlm_cache_plan against a request-by-request bookkeeping: whole numbers, so equality."""
import numpy as np
import pytest

import serve_ref as R

pytestmark = pytest.mark.gpu

NAMES = ("lens_out", "ring_state_out", "offsets", "rows", "positions", "slots", "ok")


def make(seed, n, size, most, spare, prompt=0, extra=3):
    rng = np.random.default_rng(seed)
    cap = size * most
    lens = rng.integers(0, cap + 1, n)
    fresh = np.ones(n, np.int64)
    kind = rng.random(n)
    fresh[kind < 0.2] = -1
    fresh[(kind >= 0.2) & (kind < 0.35)] = 0
    if prompt:
        long = kind > 0.7
        fresh[long] = rng.integers(1, prompt + 1, int(long.sum()))
        lens[long] = rng.integers(0, max(cap - prompt, 1), int(long.sum()))
    held = -(-lens // size)
    need = np.where((fresh > 0) & (lens + fresh <= cap), -(-(lens + fresh) // size) - held, 0)
    pool = int(held.sum() + need.sum()) + extra
    order = rng.permutation(pool)
    table = np.full((n, most), -7, np.int64)
    at = 0
    for b in range(n):
        table[b, : held[b]] = order[at: at + held[b]]
        at += held[b]
    count = min(int(need.sum() * spare), pool - at)
    head = int(rng.integers(0, pool))
    ring = np.full(pool, -5, np.int64)
    ring[(head + np.arange(count)) % pool] = order[at: at + count]
    return lens, fresh, table, ring, (head, count)


def run(lens, fresh, table, ring, state, size, tokens, in_place=False, stream=None):
    import torch

    import prng_seeded_decode_amd as S

    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    n = len(lens)
    d = dict(lens=dev(lens), fresh=dev(fresh), table=dev(table), ring=dev(ring), state=dev(state))
    out = {k: torch.full((m,), -99, dtype=torch.int32, device="cuda") for k, m in
           zip(NAMES, (n, 2, n + 1, tokens, tokens, tokens, n))}
    if in_place:
        out["lens_out"], out["ring_state_out"] = d["lens"], d["state"]
    spans = torch.full((tokens,), -99, dtype=torch.int32, device="cuda")
    S.seedlm_cache_plan(d["lens"], d["fresh"], d["table"], d["ring"], d["state"], size,
                        *(out[k] for k in NAMES), stream=stream, spans=spans)
    torch.cuda.synchronize()
    got = {k: v.cpu().tolist() for k, v in out.items()}
    assert spans.cpu().tolist() == [p + 1 if s >= 0 else 0
                                    for p, s in zip(got["positions"], got["slots"])]
    got["table"], got["ring"] = d["table"].cpu().tolist(), d["ring"].cpu().tolist()
    return got


def check(case, size, tokens, **kw):
    got, want = run(*case, size, tokens, **kw), R.plan(*case, size, tokens)
    for k in want:
        assert got[k] == want[k], k


@pytest.mark.parametrize("n,size,most,prompt,spare", [
    (1, 16, 4, 0, 1.0), (2, 1, 1, 0, 1.0), (16, 16, 32, 0, 1.0), (63, 16, 9, 40, 0.5),
    (64, 8, 20, 100, 1.0), (65, 24, 7, 30, 0.7), (513, 16, 5, 50, 0.9), (1025, 3, 6, 9, 0.6),
    (4096, 2, 3, 4, 1.0), (300, 128, 2, 200, 0.0),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_the_bookkeeping(n, size, most, prompt, spare, in_place):
    for seed in range(3):
        case = make([seed, n, size], n, size, most, spare, prompt)
        total = int(np.maximum(case[1], 0).sum())
        check(case, size, total + 5, in_place=in_place)


def test_plan_with_several_workgroups_and_in_place():
    # 30000 tokens of prompts: many workgroups, whose outputs over their inputs take a copy
    for in_place in (False, True):
        case = make([7], 200, 16, 40, 1.0, 500)
        check(case, 16, 30000, in_place=in_place)


def test_plan_with_too_few_token_entries_and_none():
    case = make([3], 40, 16, 30, 1.0, 60)
    total = int(np.maximum(case[1], 0).sum())
    for tokens in (total - 1, total // 2, 1, 0):
        check(case, 16, tokens)


def test_plan_lengths_of_zero_full_tables_and_full_pages():
    size, most = 16, 4
    lens = np.array([0, 0, 1, 15, 16, 17, 63, 64, 64, 48, 0])
    fresh = np.array([0, 1, 1, 1, 1, 15, 1, 1, 0, 16, -1])
    held = -(-lens // size)
    table = np.full((len(lens), most), -1)
    at = 0
    for b in range(len(lens)):
        table[b, : held[b]] = np.arange(at, at + held[b])
        at += held[b]
    ring = np.concatenate([np.arange(at, at + 9), np.full(at, -1)])
    for count in range(9):
        check((lens, fresh, table, ring, (0, count)), size, 64)


def test_plan_takes_wrong_lengths_and_pages_into_their_ranges():
    # lengths below 0 and above the table's, pages and queue entries outside the cache: no
    # access outside the arrays, and no slot outside the cache
    lens = np.array([-5, 1000, 20, 3])
    fresh = np.array([2, 1, 1, 1])
    table = np.array([[-1, -1], [0, 1], [2, 99], [-3, -1]])
    ring = np.array([77, 3, -2, 4, 5])
    got = run(lens, fresh, table, ring, (7, 50), 16, 6)
    want = R.plan(np.array([0, 32, 20, 3]), fresh, table, ring, (2, 5), 16, 6)
    assert got["ok"] == want["ok"] and got["slots"] == want["slots"]
    assert got["positions"] == want["positions"] and got["table"] == want["table"]
    assert all(-1 <= s < 5 * 16 for s in got["slots"])


def test_plan_on_a_strided_table_another_stream_and_a_graph():
    import torch

    import prng_seeded_decode_amd as S

    lens, fresh, table, ring, state = make([11], 24, 16, 8, 2.0, 0, extra=400)
    fresh = np.ones(24, np.int64)
    lens = np.minimum(lens, 100)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    big = torch.full((24, 13), -1, dtype=torch.int32, device="cuda")
    big[:, 2:10] = dev(table)
    d = [dev(lens), dev(fresh), big[:, 2:10], dev(ring), dev(state)]
    sizes = (25, 30, 30, 30, 24)
    outs = [torch.zeros(k, dtype=torch.int32, device="cuda") for k in sizes]
    # lengths and queue in place, as a serving loop's graph has them
    call = S.CachePlanCall(*d, 16, d[0], d[4], *outs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    now = (lens, fresh, table, ring, np.array(state))
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want = R.plan(*now, 16, 30)
        assert d[0].cpu().tolist() == want["lens_out"]
        assert d[4].cpu().tolist() == want["ring_state_out"]
        assert outs[3].cpu().tolist() == want["slots"]
        assert big[:, 2:10].cpu().tolist() == want["table"]
        now = (np.array(want["lens_out"]), fresh, np.array(want["table"]), np.array(want["ring"]),
               np.array(want["ring_state_out"]))
    assert (big[:, :2] == -1).all() and (big[:, 10:] == -1).all()


def test_plan_of_counts_whose_sums_pass_32_bits():
    # 600 requests ask for 2^31 - 1 tokens each between ones that ask for a few: those fit no
    # table, offsets stop at 2^31 - 1, and whoever comes before the first gets its pages
    big = 2 ** 31 - 1
    fresh = np.full(600, big)
    fresh[:5] = [1, 16, 0, -1, 3]
    fresh[300:310] = 2
    lens = np.zeros(600, np.int64)
    lens[3] = 20
    table = np.full((600, 4), -1)
    table[3, :2] = [9, 4]
    ring = np.array([0, 1, 2, 3, 5, 6, 7, 8, -1, -1])
    got, want = run(lens, fresh, table, ring, (0, 8), 16, 64), R.plan(lens, fresh, table, ring, (0, 8), 16, 64)
    want["offsets"] = [min(v, big) for v in want["offsets"]]
    for k in want:
        assert got[k] == want[k], k
