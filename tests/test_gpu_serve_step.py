"""The serving example's attention block over a run of steps - prompts in pieces, single tokens,
waiting and ending requests, a pool that runs out - against the same run in 64 bits.

The reference keeps every request's tokens in plain lists and knows nothing of pages.  The block
rounds to fp16 after each projection, adapter, rotation and attention (eight roundings of a
chain whose every stage is compared norm by norm), so its rows are held to 8 * 2^-11 of their
norm plus the packed projections' own documented 2e-3, twice."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "serve_attention_block", os.path.join(ROOT, "examples", "serve_attention_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def dense(m):
    import torch

    import prng_seeded_decode_amd as S

    W = torch.empty((m.rows, m.cols), dtype=torch.float32, device="cuda")
    S.seedlm_decode(m, W)
    torch.cuda.synchronize()
    return W.double().cpu().numpy()


@pytest.mark.parametrize("graph", [False, True])
def test_attention_block_over_a_run_of_steps(graph):
    import torch

    import prng_seeded_decode_amd as S
    from workloads import gen_records

    E = example()
    hidden, heads, kv, dim, requests, rows, size = 256, 4, 2, 64, 5, 8, 4
    mats = [S.seedlm_pack(*gen_records(6, i, r, c, 8, 3), r, c, 8, 3, 16)
            for i, (r, c) in enumerate(((heads * dim, hidden), (kv * dim, hidden),
                                        (kv * dim, hidden), (hidden, heads * dim)))]
    block = E.AttentionBlock(mats, heads, kv, dim, requests, pages=11, rows=rows, page_size=size,
                             max_pages=6, adapters=3, rank=8)
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

    rng = np.random.default_rng(12)
    keys, values = [[] for _ in range(requests)], [[] for _ in range(requests)]
    free = 11
    script = [[3, 1, 0, 2, 2], [1, 1, 4, 1, 1], [1, 1, 1, 1, 1], [1, 1, 1, -1, 1], [0, 1, 1, 3, 1],
              [5, 0, 1, 1, 1], [1, 1, 1, 1, 1], [1, -1, 1, 1, 1], [1, 6, 1, 0, 0], [1, 1, 1, 1, 1],
              [2, 2, 2, 2, 0], [1, 1, 1, 1, 1]]
    refused = 0
    for step, fresh in enumerate(script):
        x = rng.standard_normal((rows, hidden)).astype(np.float16)
        block.x.copy_(torch.from_numpy(x))
        block.fresh.copy_(torch.tensor(fresh, dtype=torch.int32))
        block.step()
        torch.cuda.synchronize()
        got, ok = block.out.double().cpu().numpy(), block.ok.cpu().tolist()
        who = np.full(rows, -1)
        owner, t, wanted, returned = [], 0, 0, 0
        for b, n in enumerate(fresh):
            length = len(keys[b])
            if n < 0:
                returned += -(-length // size)
                keys[b], values[b] = [], []
                assert ok[b] == 1
                continue
            need = -(-(length + n) // size) - -(-length // size)
            fits = length + n <= 6 * size and t + n <= rows
            wanted += need if fits else 0
            granted = fits and (need == 0 or wanted <= free)
            assert ok[b] == int(granted), (step, b)
            refused += not granted
            for i in range(n):
                if t + i < rows:
                    owner.append((t + i, b, length + i, granted))
                    who[t + i] = adapters[b]
            t += n
        free = int(block.ring_state[1])
        qkv = [project(i, x.astype(np.float64), who) for i in range(3)]
        mixed = np.zeros((rows, heads * dim))
        for row, b, pos, granted in owner:
            if granted:
                keys[b].append(turn(qkv[1][row].reshape(kv, dim), pos))
                values[b].append(qkv[2][row].reshape(kv, dim))
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
            err = np.linalg.norm(got[row] - want[row])
            if granted:
                assert err <= (8 * 2.0 ** -11 + 4e-3) * np.linalg.norm(want[row]), (step, row, err)
        for row in range(rows):
            if row not in [o[0] for o in owner if o[3]]:
                assert (got[row] == 0).all()
    assert refused > 0
    assert block.lens.cpu().tolist() == [len(k) for k in keys]


def test_example_runs():
    import subprocess
    import sys

    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "serve_attention_block.py"),
                        "--config", "3", "--requests", "4", "--steps", "20"],
                       capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "us a step" in r.stdout
