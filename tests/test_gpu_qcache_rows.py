"""seedlm_qcache_attend with `rows`, as a serving plan hands them over: one token of each request,
pieces of prompts, both in one batch, and padding, through one call whose sizes stay."""
import numpy as np
import pytest

from test_gpu_qcache_attend import check, make, run, run_rows, widen

pytestmark = pytest.mark.gpu

# heads, cache heads, dimensions, bits, groups: several queries an item at most, and one (16 heads
# of a cache head)
FORMS = [(8, 2, 128, 4, 1), (4, 4, 64, 8, 2), (16, 2, 256, 4, 1), (16, 1, 128, 4, 2)]


def call_of(x, q, rows, lens, out):
    import torch

    import prng_seeded_decode_amd as S

    i32 = lambda a: torch.tensor([int(v) for v in a], dtype=torch.int32, device="cuda")
    return S.QCacheAttendCall(q, *x["cache"], x["dtable"], i32(lens), out,
                              rows=None if rows is None else i32(rows))


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("heads,kv,dim,bits,groups", FORMS)
@pytest.mark.parametrize("n", [1, 5, 63, 64, 65, 150])
@pytest.mark.parametrize("pages", [0, 700])
def test_one_token_a_request_is_the_call_without_rows(pages, n, heads, kv, dim, bits, groups, f16):
    # the same split of the same work, whole (most of the narrow tables) and in runs: the same bits
    import torch

    rng = np.random.default_rng([n, dim])
    lens = [int(v) for v in np.exp(rng.uniform(0, np.log(700), n)).astype(int) * rng.integers(0, 4, n).clip(0, 1)]
    lens[n // 2] = 600
    x = make([n, dim], lens, heads, kv, dim, 16, f16, bits, groups)
    if pages:
        x = widen(x, pages)
    plain = run(x)
    check(x, plain)
    assert np.array_equal(run_rows(x, x["dq"], range(n), lens), plain)
    out = torch.empty_like(x["dq"])
    need = [call_of(x, x["dq"], rows, lens, out).scratch_bytes() for rows in (None, range(n))]
    assert need[0] == need[1] and (need[0] > 0 or pages == 0)


@pytest.mark.parametrize("heads,kv,dim,bits,groups", FORMS)
@pytest.mark.parametrize("n", [11, 64, 70])
@pytest.mark.parametrize("pages", [0, 700])
def test_batches_of_single_tokens_pieces_and_padding(pages, n, heads, kv, dim, bits, groups):
    # a captured call takes each of the plans in turn: its sizes are all that it was made for
    import torch

    import prng_seeded_decode_amd as S

    held = [300, 40, 600, 129, 17, 1, 128, 0]
    x = make([n, dim, 3], held, heads, kv, dim, 16, True, bits, groups)
    if pages:
        x = widen(x, pages)
    rng = np.random.default_rng(n)
    plans = [
        [i % 8 for i in range(n)],                                 # nothing is shared
        [i * 8 // n for i in range(n)],                            # pieces
        [0, 1, 2] + [3] * (n - 8) + [4, 5, 6] + [-1] * 2,          # single tokens about a piece
        [2] * n,
        [-1] * n,
        [2, -1] * (n // 2) + [2] * (n % 2),
        sorted(int(r) for r in rng.integers(-1, 9, n)),            # 8 is outside the table too
        [int(r) for r in rng.integers(-1, 9, n)],
        list(range(8)) + [7] * (n - 8),
    ]
    g = torch.Generator(device="cuda").manual_seed(n)
    q = torch.randn((n, heads, dim), generator=g, device="cuda").half()
    host = q.cpu().numpy()
    out = torch.empty_like(q)
    drows = torch.zeros(n, dtype=torch.int32, device="cuda")
    dlens = torch.zeros(n, dtype=torch.int32, device="cuda")
    call = S.QCacheAttendCall(q, *x["cache"], x["dtable"], dlens, out, rows=drows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()  # the stream's scratch exists before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for plan in plans:
        assert len(plan) == n
        most = [held[r] if 0 <= r < 8 else 9 for r in plan]
        lens = [int(rng.integers(0, m + 1)) if i % 3 else m for i, m in enumerate(most)]
        drows.copy_(torch.tensor(plan, dtype=torch.int32))
        dlens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        check(x, got, lens=lens, rows=plan, q=host)
        assert np.array_equal(got, run_rows(x, q, plan, lens))
