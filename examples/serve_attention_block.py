"""One decoder layer's attention block, served from packed weights for a batch of requests.

    python examples/serve_attention_block.py [--config 3] [--requests 16] [--steps 64]

Every step: page tables, positions and slots from the requests' lengths
(seedlm_cache_plan); the packed q, k and v projections (seedlm_gemv_many) with each request's
adapter beside them (seedlm_lora_many); rotary positions and the cache write
(seedlm_cache_append); attention over the pages (seedlm_cache_attend); the packed o projection
and its adapters.  All buffers are made once and every call is marshalled once, so a step is a
fixed list of launches and is captured into a HIP graph; lengths, pages and adapters only
change on the GPU.  Weights, adapters and inputs are synthetic.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import prng_seeded_decode_amd as S  # noqa: E402
from workloads import CONFIGS, gen_records  # noqa: E402


class AttentionBlock:
    """q, k, v and o as packed matrices, adapters for each, and a paged cache.

    `requests` requests share `rows` activation rows a step.  `fresh` (int32 [requests]) says
    how many of the next rows each request takes: 1 for the next token, more for a piece of a
    prompt, 0 to wait, -1 to end.  `x` (fp16 [rows][hidden]) holds those rows one request
    after another, and `out` gets theirs; rows past the last one come out as zeros.
    `adapter` (int32 [requests]) names each request's adapter, -1 for none."""

    def __init__(self, mats, heads, kv_heads, dim, requests, pages, rows=None, page_size=16,
                 max_pages=64, adapters=4, rank=16, theta=500000.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        f16 = dict(dtype=torch.float16, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        q, k, v, o = mats
        if q.rows != heads * dim or k.rows != kv_heads * dim or v.rows != k.rows or o.cols != q.rows:
            raise ValueError("the matrices do not fit the heads")
        n = rows = requests if rows is None else rows
        self.mats = mats
        self.x = torch.zeros((n, q.cols), **f16)
        self.q, self.k, self.v = (torch.empty((n, m.rows), **f16) for m in (q, k, v))
        self.mixed, self.out = torch.empty((n, q.rows), **f16), torch.empty((n, o.rows), **f16)

        # the serving state, per request
        self.lens, self.fresh = torch.zeros(requests, **i32), torch.ones(requests, **i32)
        self.table = torch.full((requests, max_pages), -1, **i32)
        self.ring = torch.arange(pages, **i32)
        self.ring_state = torch.tensor([0, pages], **i32)
        self.ok = torch.zeros(requests, **i32)
        self._adapter = torch.full((requests + 1,), -1, **i32)  # the last one for idle rows
        self.adapter = self._adapter[:requests]
        # and per row
        offsets = torch.zeros(requests + 1, **i32)
        self.rows, self.positions, self.slots, self.spans, self.row_adapter = (
            torch.zeros(n, **i32) for _ in range(5))
        self.k_cache = torch.zeros((pages, page_size, kv_heads, dim), **f16)
        self.v_cache = torch.zeros_like(self.k_cache)
        inv = theta ** (-torch.arange(dim // 2, dtype=torch.float64, device="cuda") * 2 / dim)
        angle = torch.arange(max_pages * page_size, device="cuda")[:, None] * inv
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        self.scales = torch.ones(adapters, device="cuda")
        self.A = [torch.randn((adapters, rank, m.cols), generator=g, device="cuda")
                  .mul(m.cols ** -0.5).half() for m in mats]
        self.B = [torch.randn((adapters, m.rows, rank), generator=g, device="cuda")
                  .mul(0.1 * rank ** -0.5).half() for m in mats]

        heads_of = lambda t, h: t.view(n, h, dim)
        site = lambda i, x, y: (x, self.A[i], self.B[i], y, y)
        plan = S.CachePlanCall(self.lens, self.fresh, self.table, self.ring, self.ring_state,
                               page_size, self.lens, self.ring_state, offsets, self.rows,
                               self.positions, self.slots, self.ok, spans=self.spans)
        # row -1 reads the entry for idle rows
        adapters_of_rows = lambda: self.row_adapter.copy_(self._adapter[self.rows.long()])
        self.calls = [
            plan,
            adapters_of_rows,
            S.GemvManyCall([q, k, v], [self.x] * 3, [self.q, self.k, self.v], batch=n),
            S.LoraCall([site(0, self.x, self.q), site(1, self.x, self.k), site(2, self.x, self.v)],
                       self.row_adapter, self.scales),
            S.CacheAppendCall(heads_of(self.q, heads), heads_of(self.k, kv_heads),
                              heads_of(self.v, kv_heads), self.cos, self.sin, self.positions,
                              self.slots, heads_of(self.q, heads), self.k_cache, self.v_cache),
            S.CacheAttendCall(heads_of(self.q, heads), self.k_cache, self.v_cache, self.table,
                              self.spans, heads_of(self.mixed, heads), rows=self.rows),
            S.GemvManyCall([o], [self.mixed], [self.out], batch=n),
            S.LoraCall([site(3, self.mixed, self.out)], self.row_adapter, self.scales),
        ]
        self.graph = None

    def step(self):
        """Enqueue one step on torch's current stream (or replay the captured one)."""
        if self.graph is not None:
            self.graph.replay()
            return
        for call in self.calls:
            call()

    def capture(self):
        """Capture the step.  A step in which all requests wait runs first, so that the
        stream's scratch exists; it leaves the serving state as it is."""
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            fresh = self.fresh.clone()
            self.fresh.zero_()
            self.step()
            self.fresh.copy_(fresh)
        torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            self.step()
        self.graph = graph


def packed_layer(config):
    """The config's q, k, v and o with synthetic records, and its heads."""
    c = CONFIGS[config]
    mats = []
    for i, m in enumerate(c.matrices[:4]):
        mats.append(S.seedlm_pack(*gen_records(config, i, m.rows, m.cols, c.C, c.P), m.rows, m.cols,
                                  c.C, c.P, c.K))
    dim = 128
    return mats, mats[0].rows // dim, mats[1].rows // dim, dim


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--config", type=int, default=3, choices=(2, 3, 4), help="layer of workloads.CONFIGS")
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--steps", type=int, default=64)
    args = ap.parse_args()
    if not 1 <= args.requests <= S.MAX_BATCH:
        ap.error(f"--requests must be 1 to {S.MAX_BATCH}")
    mats, heads, kv_heads, dim = packed_layer(args.config)
    n = args.requests
    # one token a step, so a step's rows are the requests
    max_pages = -(-(args.steps + 2) // 16) + 1
    block = AttentionBlock(mats, heads, kv_heads, dim, n, n * max_pages, max_pages=max_pages)
    block.adapter.copy_(torch.arange(n) % 4)
    block.capture()
    block.step()
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(args.steps):
        block.x.normal_()
        block.step()
    torch.cuda.synchronize()
    each = (time.perf_counter() - begin) / args.steps
    if not bool(block.out.isfinite().all()) or int(block.lens.min()) != args.steps + 1:
        raise SystemExit("the steps did not give what they should")
    print(f"{CONFIGS[args.config].name}: attention block of {n} requests, {args.steps} steps, "
          f"{each * 1e6:.1f} us a step")


if __name__ == "__main__":
    main()
