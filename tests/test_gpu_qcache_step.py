"""The quantised cache in use: the serving example's attention block over a run of steps - prompts in
pieces, single tokens, waiting and ending requests, a pool that runs out - with its cache in 4 and
8 bits.

The reference keeps every request's tokens in plain lists and knows nothing of pages.  What it
appends is compared with what the block's cache holds of the same token (read back by
seedlm_qcache_read): half a step, the rounding of the step, and the block's own fp16 roundings
before it.  Its attention then goes on with what the cache holds, so that its rows are held to the
bound of the fp16 block: 8 * 2^-11 of their norm plus the packed projections' documented 2e-3,
twice."""
import os
import subprocess
import sys

import numpy as np
import pytest

import qcache_ref as Q
from test_gpu_serve_step import ROOT, dense, example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,groups", [(4, 2), (8, 1)])
@pytest.mark.parametrize("graph", [False, True])
def test_attention_block_on_a_quantised_cache(graph, bits, groups):
    import torch

    import prng_seeded_decode_amd as S
    from workloads import gen_records

    E = example()
    hidden, heads, kv, dim, requests, rows, size = 256, 4, 2, 64, 5, 8, 4
    mats = [S.seedlm_pack(*gen_records(6, i, r, c, 8, 3), r, c, 8, 3, 16)
            for i, (r, c) in enumerate(((heads * dim, hidden), (kv * dim, hidden),
                                        (kv * dim, hidden), (hidden, heads * dim)))]
    block = E.AttentionBlock(mats, heads, kv, dim, requests, pages=11, rows=rows, page_size=size,
                             max_pages=6, adapters=3, rank=8, cache_bits=bits, groups=groups)
    W = [dense(m) for m in mats]
    A = [t.double().cpu().numpy() for t in block.A]
    B = [t.double().cpu().numpy() for t in block.B]
    cos, sin = block.cos.double().cpu().numpy(), block.sin.double().cpu().numpy()
    adapters = np.array([0, -1, 2, 1, 0])
    block.adapter.copy_(torch.from_numpy(adapters.astype(np.int32)))
    if graph:
        block.capture()

    def project(i, x, who):
        y = x @ W[i].T
        for t, a in enumerate(who):
            if a >= 0:
                y[t] += B[i][a] @ (A[i][a] @ x[t])
        return y

    def turn(v, pos):
        half = dim // 2
        a, b, c, s = v[:, :half], v[:, half:], cos[pos], sin[pos]
        return np.concatenate([a * c - b * s, b * c + a * s], 1)

    backs = [torch.zeros((rows, kv, dim), device="cuda") for _ in range(2)]
    read = S.QCacheReadCall(*block.cache, block.slots, *backs)
    rng = np.random.default_rng(12)
    keys, values = [[] for _ in range(requests)], [[] for _ in range(requests)]
    script = [[3, 1, 0, 2, 2], [1, 1, 4, 1, 1], [1, 1, 1, 1, 1], [1, 1, 1, -1, 1], [0, 1, 1, 3, 1],
              [5, 0, 1, 1, 1], [1, 1, 1, 1, 1], [1, -1, 1, 1, 1], [1, 6, 1, 0, 0], [1, 1, 1, 1, 1],
              [2, 2, 2, 2, 0], [1, 1, 1, 1, 1]]
    refused = 0
    for step, fresh in enumerate(script):
        x = rng.standard_normal((rows, hidden)).astype(np.float16)
        block.x.copy_(torch.from_numpy(x))
        block.fresh.copy_(torch.tensor(fresh, dtype=torch.int32))
        block.step()
        read()
        torch.cuda.synchronize()
        got, ok = block.out.double().cpu().numpy(), block.ok.cpu().tolist()
        held = [t.double().cpu().numpy() for t in backs]
        slots = block.slots.cpu().numpy()
        steps = [p.cpu().numpy()[slots // size, slots % size][..., 0].astype(np.float64)
                 for p in block.cache[2:]]
        who, owner, t = np.full(rows, -1), [], 0
        for b, n in enumerate(fresh):
            if n < 0:
                keys[b], values[b] = [], []
                continue
            refused += not ok[b]
            for i in range(n):
                if t + i < rows:
                    owner.append((t + i, b, len(keys[b]) + i, ok[b]))
                    who[t + i] = adapters[b]
            t += n
        qkv = [project(i, x.astype(np.float64), who) for i in range(3)]
        mixed = np.zeros((rows, heads * dim))
        for row, b, pos, granted in owner:
            if not granted:
                assert slots[row] == -1 and not held[0][row].any()
                continue
            for j, (store, ref) in enumerate(((keys, turn(qkv[1][row].reshape(kv, dim), pos)),
                                              (values, qkv[2][row].reshape(kv, dim)))):
                s = steps[j][row].repeat(dim // groups, -1)
                tol = s / 2 + (2 ** bits - 1) * np.maximum(s * 2.0 ** -11, 2.0 ** -25)
                tol += (4 * 2.0 ** -11 + 4e-3) * np.linalg.norm(ref)
                assert np.all(np.abs(held[j][row] - ref) <= tol), (step, row, j)
                store[b].append(held[j][row])
        for row, b, pos, granted in owner:
            if not granted:
                continue
            q = turn(qkv[0][row].reshape(heads, dim), pos)
            for h in range(heads):
                k = np.array([v[h // 2] for v in keys[b][: pos + 1]])
                v = np.array([v[h // 2] for v in values[b][: pos + 1]])
                s = k @ q[h] * dim ** -0.5
                p = np.exp(s - s.max())
                mixed[row, h * dim: (h + 1) * dim] = p @ v / p.sum()
        want = project(3, mixed, who)
        for row, b, pos, granted in owner:
            if granted:
                err = np.linalg.norm(got[row] - want[row])
                assert err <= (8 * 2.0 ** -11 + 4e-3) * np.linalg.norm(want[row]), (step, row, err)
        for row in range(rows):
            if row not in [o[0] for o in owner if o[3]]:
                assert (got[row] == 0).all()
    assert refused > 0
    assert block.lens.cpu().tolist() == [len(k) for k in keys]


@pytest.mark.parametrize("bits", ["4", "8"])
def test_example_runs_on_a_quantised_cache(bits):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "serve_attention_block.py"),
                        "--config", "3", "--requests", "4", "--steps", "20", "--cache-bits", bits],
                       capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "us a step" in r.stdout


def attention(seed, lens, heads=8, kv=2, dim=128, size=16, bits=4, groups=2):
    """Random codes and pairs in pages in order, and a call over them."""
    import torch

    import prng_seeded_decode_amd as S

    g = torch.Generator(device="cuda").manual_seed(seed)
    n, most = len(lens), -(-max(lens) // size)
    codes = [torch.randint(0, 256, (n * most, size, kv, dim * bits // 8), generator=g, device="cuda",
                           dtype=torch.uint8) for _ in range(2)]
    pairs = [torch.rand((n * most, size, kv, groups, 2), generator=g, device="cuda").half() * 0.1
             for _ in range(2)]
    q = torch.randn((n, heads, dim), generator=g, device="cuda").half()
    table = torch.arange(n * most, dtype=torch.int32, device="cuda").view(n, most)
    out = torch.zeros_like(q)
    i32 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return S.QCacheAttendCall(q, *codes, *pairs, table, i32, out), out


def test_calls_on_two_streams_and_two_graphs_side_by_side():
    import torch

    calls = [attention(i, [3000 + 700 * i, 1, 0, 900]) for i in range(2)]
    want = []
    for call, out in calls:
        assert call.scratch_bytes() > 0
        call()
        torch.cuda.synchronize()
        want.append(out.clone())
    streams = [torch.cuda.Stream() for _ in calls]
    for (call, _), s in zip(calls, streams):
        call(stream=s)  # the streams' scratch
    torch.cuda.synchronize()
    for _ in range(10):
        for (call, out), s in zip(calls, streams):
            with torch.cuda.stream(s):
                out.zero_()
            call(stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(out, w) for (_, out), w in zip(calls, want))
    graphs = []
    for (call, _), s in zip(calls, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            call()
    for _ in range(6):
        for _, out in calls:
            out.fill_(3.0)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        calls[0][0](stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        assert all(torch.equal(out, w) for (_, out), w in zip(calls, want))


def test_a_read_back_equals_the_definition_after_appends_to_shared_pages():
    # rows of one page written by two calls keep to their own bytes
    import torch

    import prng_seeded_decode_amd as S

    g = torch.Generator(device="cuda").manual_seed(3)
    kv, dim, size, bits = 3, 64, 8, 4
    cache = [torch.zeros((2, size, kv, dim * bits // 8), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.zeros((2, size, kv, 1, 2), dtype=torch.float16, device="cuda") for _ in range(2)]
    table = torch.ones((4, 0), device="cuda"), torch.zeros((4, 0), device="cuda")
    x = torch.randn((16, kv, dim), generator=g, device="cuda").half()
    pos = torch.zeros(16, dtype=torch.int32, device="cuda")
    slots = torch.randperm(16, generator=g, device="cuda").int()
    for part in (slice(0, 5), slice(5, 16)):
        n = len(range(16)[part])
        q = torch.zeros((n, kv, dim), dtype=torch.float16, device="cuda")
        S.seedlm_qcache_append(q, x[part], -x[part], *table, pos[part], slots[part], q, *cache)
    outs = [torch.zeros((16, kv, dim), device="cuda") for _ in range(2)]
    S.seedlm_qcache_read(*cache, slots, *outs)
    for got, src in zip(outs, (x, -x)):
        rows, pairs = Q.quantise(src.cpu().numpy(), bits, dim)
        assert np.array_equal(got.cpu().numpy(), Q.values(rows, pairs, bits)[0].astype(np.float32))
