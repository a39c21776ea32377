"""Cases of the serving operators on a quantised cache: writing it, reading it back, and
attention over it.

Every case runs in two forms.  The plain form is written from the formulas in elementary torch
operations, in 32 bits, rounded once at the end; the other makes the library's calls.  `exact`
gives the same outputs from the definitions in 64 bits.

    store   rotary positions on q and k, k and v quantised into their cache slots, and what the
            cache then holds read back, as a prompt's own attention uses it
    read    tokens of the cache read back
    attend  query tokens over their requests' pages of the cache

A cache row (one token of one head) is `dim` codes of 4 or 8 bits: 16 units of dim / 16 codes,
unit w holding elements w, w + 16, w + 32, ... from its lowest bits up.  Each `group`
consecutive elements share an fp16 pair (scale, offset), code c standing for
offset + scale * c.
"""
import math

import numpy as np
import torch

own = False

_F = {"f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # A piece of 16 new tokens with the Llama-3-70B layer's heads: latency.
        {"name": "store_piece_16", "op": "store", "tokens": 16, "heads": 64, "kv_heads": 8,
         "dim": 128, "rot": 128, "interleaved": False, "dtype": "f16", "bits": 4, "group": 64,
         "page_size": 16, "pages": 1024, "head_major": True},
        # A prompt of odd length with the Llama-2-7B layer's heads, 4 bits.
        {"name": "store_prompt_4097", "op": "store", "tokens": 4097, "heads": 32, "kv_heads": 32,
         "dim": 128, "rot": 128, "interleaved": False, "dtype": "f16", "bits": 4, "group": 128,
         "page_size": 16, "pages": 512, "head_major": True},
        # fp32 activations, 64 dimensions of which half turn as interleaved pairs, 8 bits, small
        # groups, an odd number of tokens, token-major pages of 24.
        {"name": "store_f32_515", "op": "store", "tokens": 515, "heads": 32, "kv_heads": 8,
         "dim": 64, "rot": 32, "interleaved": True, "dtype": "f32", "bits": 8, "group": 32,
         "page_size": 24, "pages": 100, "head_major": False},
        # One short request read back from an 8-bit cache: latency.
        {"name": "read_one_300", "op": "read", "tokens": 300, "kv_heads": 8, "dim": 128,
         "dtype": "f32", "bits": 8, "group": 128, "page_size": 16, "pages": 64,
         "head_major": True},
        # A long request's 4-bit tokens back as fp16, to leave the cache: bandwidth.
        {"name": "read_32771", "op": "read", "tokens": 32771, "kv_heads": 8, "dim": 128,
         "dtype": "f16", "bits": 4, "group": 64, "page_size": 16, "pages": 2100,
         "head_major": True},
        # One short request on the Llama-3-8B layer's heads: latency.
        {"name": "attend_one_300", "op": "attend", "requests": 1, "per": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "max_len": 300, "ragged": False, "dtype": "f16", "bits": 4,
         "group": 128, "page_size": 16, "head_major": True},
        # 16 ragged requests (an empty and a one-token one among them), Llama-3-70B heads.
        {"name": "attend_ragged_16", "op": "attend", "requests": 16, "per": 1, "heads": 64,
         "kv_heads": 8, "dim": 128, "max_len": 8192, "ragged": True, "dtype": "f16", "bits": 4,
         "group": 64, "page_size": 16, "head_major": True},
        # fp32 queries and outputs, no shared heads, 64 dimensions, 8 bits, pages of 64.
        {"name": "attend_f32_8", "op": "attend", "requests": 8, "per": 1, "heads": 32,
         "kv_heads": 32, "dim": 64, "max_len": 2047, "ragged": True, "dtype": "f32", "bits": 8,
         "group": 64, "page_size": 64, "head_major": True},
        # Pieces of four prompts, 128 new tokens each behind what is cached already.
        {"name": "attend_pieces_4x128", "op": "attend", "requests": 4, "per": 128, "heads": 32,
         "kv_heads": 8, "dim": 128, "max_len": 2100, "ragged": True, "dtype": "f16", "bits": 4,
         "group": 32, "page_size": 16, "head_major": False},
        # 256 dimensions in 8 bits, few heads, token-major pages.
        {"name": "attend_dim256_12", "op": "attend", "requests": 12, "per": 1, "heads": 16,
         "kv_heads": 4, "dim": 256, "max_len": 5000, "ragged": True, "dtype": "f16", "bits": 8,
         "group": 128, "page_size": 16, "head_major": False},
        # One very long request: the work has to be split over the cache's length.
        {"name": "attend_one_131071", "op": "attend", "requests": 1, "per": 1, "heads": 64,
         "kv_heads": 8, "dim": 128, "max_len": 131071, "ragged": False, "dtype": "f16", "bits": 4,
         "group": 128, "page_size": 16, "head_major": True},
        # A full batch of long ragged requests, Llama-3-8B heads: bandwidth.
        {"name": "attend_ragged_64", "op": "attend", "requests": 64, "per": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "max_len": 16384, "ragged": True, "dtype": "f16", "bits": 4,
         "group": 128, "page_size": 32, "head_major": True},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "store", "read", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    bits = rng.choice([4, 4, 8])
    group = dim // rng.choice([1, 2] if dim == 64 else [1, 2, 4])
    dtype = rng.choice(["f16", "f16", "f32"])
    width = 4 if dtype == "f32" else 2
    size = rng.choice([1, 16, 16, 24, 64, 256])
    head_major = rng.random() < 0.6
    same = {"dim": dim, "dtype": dtype, "bits": bits, "group": group, "page_size": size,
            "head_major": head_major}
    kv = rng.choice([1, 2, 4, 8, 8, 32])
    if op == "store":
        heads = kv * rng.choice([1, 4] if kv > 4 else [1, 4, 8])
        tokens = _log(rng, 1, min(16384, 4097 * 96 * 256 // ((heads + 2 * kv) * dim * width)))
        return {"op": op, "tokens": tokens, "heads": heads, "kv_heads": kv, "rot": rng.choice([dim, dim, dim // 2]),
                "interleaved": rng.random() < 0.4, "pages": -(-tokens // size) + _log(rng, 1, 512), **same}
    if op == "read":
        tokens = _log(rng, 1, min(2 ** 17, 32771 * 8 * 256 // (kv * dim * width)))
        return {"op": op, "tokens": tokens, "kv_heads": kv,
                "pages": -(-tokens // size) + _log(rng, 1, 512), **same}
    heads = kv * rng.choice([1, 2, 4, 6, 8])
    requests, per = _log(rng, 1, 64), 1
    if rng.random() < 0.25:  # pieces of prompts
        requests = min(requests, 8)
        per = _log(rng, 2, max(2, min(128, 2 ** 21 // (requests * heads * dim))))
    most = min(131071, int(3.4e9) // (requests * kv * dim * bits),
               int(2.2e9) // (requests * per * heads * dim))
    return {"op": op, "requests": requests, "per": per, "heads": heads, "kv_heads": kv,
            "max_len": _log(rng, per, max(most, per + 1)),
            "ragged": requests > 1 and rng.random() < 0.8, **same}


# ---- inputs ----


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed)), np.random.default_rng(int(seed))


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _pools(case, g, pages):
    """Codes [pages][page_size][kv_heads][bytes of a row] and pairs [pages][page_size][kv_heads]
    [groups][2] of keys and of values, as earlier requests left them; head_major: stored with the
    heads outside of a page's tokens."""
    size, kv, dim = case["page_size"], case["kv_heads"], case["dim"]
    outer = (pages, kv, size) if case["head_major"] else (pages, size, kv)
    levels = 2 ** case["bits"] - 1
    pools = []
    for spread in (6.0, 3.0):
        codes = torch.randint(0, 256, (*outer, dim * case["bits"] // 8), generator=g, device="cuda",
                              dtype=torch.uint8)
        shape = (*outer, dim // case["group"])
        scale = (0.5 + torch.rand(shape, generator=g, device="cuda")) * (spread / levels)
        offset = -scale * (levels / 2) + 0.2 * torch.randn(shape, generator=g, device="cuda")
        pools += [codes, torch.stack([scale, offset], -1).half()]
    if case["head_major"]:
        pools = [p.transpose(1, 2) for p in pools]
    k, ks, v, vs = pools
    return {"k_cache": k, "v_cache": v, "k_scale": ks, "v_scale": vs}


def _prepare_store(case, g, rng):
    t, dim, dt = case["tokens"], case["dim"], _F[case["dtype"]]
    size, pages, kv = case["page_size"], case["pages"], case["kv_heads"]
    last = 8192
    slots = rng.permutation(size * pages)[:t]
    slots[1:][rng.random(t - 1) < 0.02] = -1  # padding rows
    angle = torch.arange(last, device="cuda", dtype=torch.float64)[:, None] * (
        10000.0 ** (-torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
                    * 2 / case["rot"]))
    # keys have a few channels that are far larger than the others
    wide = 1.0 + 6.0 * (torch.rand((kv, dim), generator=g, device="cuda") < 0.03).float()
    state = {"q": _randn(g, (t, case["heads"], dim), dt),
             "k": (torch.randn((t, kv, dim), generator=g, device="cuda") * wide).to(dt),
             "v": _randn(g, (t, kv, dim), dt),
             "cos": angle.cos().float(), "sin": angle.sin().float(),
             "positions": _ints(rng.integers(0, last, t)), "slots": _ints(slots),
             "q_out": torch.zeros((t, case["heads"], dim), dtype=dt, device="cuda"),
             "k_back": torch.zeros((t, kv, dim), dtype=torch.float16, device="cuda"),
             "v_back": torch.zeros((t, kv, dim), dtype=torch.float16, device="cuda")}
    return {**state, **_pools(case, g, pages)}


def _prepare_read(case, g, rng):
    t, dim, dt = case["tokens"], case["dim"], _F[case["dtype"]]
    size, pages = case["page_size"], case["pages"]
    order = rng.permutation(pages)
    at = np.arange(t)
    slots = order[at // size] * size + at % size
    shape = (t, case["kv_heads"], dim)
    return {"slots": _ints(slots), "k_out": torch.zeros(shape, dtype=dt, device="cuda"),
            "v_out": torch.zeros(shape, dtype=dt, device="cuda"), **_pools(case, g, pages)}


def _prepare_attend(case, g, rng):
    n, per, size, top, dim = (case[k] for k in ("requests", "per", "page_size", "max_len", "dim"))
    ends = np.full(n, top)
    if case["ragged"]:
        ends = rng.integers(per, top + 1, n)
        ends[: 3] = [top, 0 if per == 1 else per, per][: min(n, 3)]
        ends = rng.permutation(ends)
    held = -(-ends // size)
    most = -(-top // size)
    pages = int(held.sum()) + 2
    order = rng.permutation(pages)
    table = np.full((n, most), -1, np.int64)
    at = np.concatenate([[0], np.cumsum(held)])
    for b in range(n):
        table[b, : held[b]] = order[at[b]: at[b + 1]]
    dt = _F[case["dtype"]]
    # a request's queries are its last tokens, each of which sees those up to itself
    lens = ends[:, None] - per + 1 + np.arange(per)[None, :]
    state = {"q": _randn(g, (n * per, case["heads"], dim), dt, 1.5), "table": _ints(table),
             "lens": _ints(np.maximum(lens, 0).reshape(-1)), "scale": dim ** -0.5,
             "rows": _ints(np.repeat(np.arange(n), per)) if per > 1 else None,
             "out": torch.zeros((n * per, case["heads"], dim), dtype=dt, device="cuda")}
    return {**state, **_pools(case, g, pages)}


def prepare(case, seed):
    g, rng = _gen(seed)
    make = {"store": _prepare_store, "read": _prepare_read, "attend": _prepare_attend}
    return {"case": dict(case), **make[case["op"]](case, g, rng)}


# ---- the plain forms ----


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    head, tail = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, tail], -1)


def _quantise(x, bits, group):
    """Codes [..., dim], and scale and offset [..., groups], of fp16 values."""
    x = x.float().unflatten(-1, (-1, group))
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    # one division of two numbers of at most 12 bits: 32 bits decide as 64 would
    scale = ((high - low) / (2 ** bits - 1)).half()
    step = scale.float()
    code = torch.round((x - low) / torch.where(step == 0, torch.ones_like(step), step))
    code = torch.where(step == 0, torch.zeros_like(code), code.clamp(0, 2 ** bits - 1))
    return code.flatten(-2), scale[..., 0], low[..., 0].half()


def _pack(code, bits):
    """Codes [..., dim] as the bytes of a row."""
    units = code.to(torch.uint8).unflatten(-1, (-1, 16)).transpose(-1, -2)
    if bits == 4:
        units = units[..., 0::2] | (units[..., 1::2] << 4)
    return units.flatten(-2)


def _unpack(rows, bits):
    """The codes [..., dim] of rows' bytes, as fp32."""
    units = rows.unflatten(-1, (16, -1))
    if bits == 4:
        units = torch.stack([units & 15, units >> 4], -1).flatten(-2)
    return units.transpose(-1, -2).flatten(-2).float()


def _values(rows, pairs, bits):
    """What rows [..., bytes] with pairs [..., groups, 2] stand for, in fp32."""
    code = _unpack(rows, bits)
    code = code.unflatten(-1, (pairs.shape[-2], -1))
    return (pairs[..., 1:].float() + pairs[..., :1].float() * code).flatten(-2)


def _at(slots, size):
    slots = slots.long()
    return slots // size, slots % size


def _plain_store(s):
    case = s["case"]
    bits, group, rot, inter = case["bits"], case["group"], case["rot"], case["interleaved"]
    pos = s["positions"].long()
    cos, sin = s["cos"][pos][:, None, :], s["sin"][pos][:, None, :]
    q = _rotate(s["q"], cos, sin, rot, inter).to(s["q"].dtype)
    # padding rows (slot -1) write once more what row 0, never one of them, writes
    keep = (s["slots"] >= 0)[:, None, None]
    at = _at(torch.where(keep[:, 0, 0], s["slots"], s["slots"][:1]), case["page_size"])

    def put(x, cache, pairs):
        code, scale, offset = _quantise(x.half(), bits, group)
        row, pair = _pack(code, bits), torch.stack([scale, offset], -1)
        cache[at] = torch.where(keep, row, row[:1])
        pairs[at] = torch.where(keep[..., None], pair, pair[:1])
        return torch.where(keep, _values(row, pair, bits), torch.zeros_like(code)).half()

    k_back = put(_rotate(s["k"], cos, sin, rot, inter), s["k_cache"], s["k_scale"])
    v_back = put(s["v"], s["v_cache"], s["v_scale"])
    return [q, k_back, v_back, s["k_scale"], s["v_scale"]]


def _plain_read(s):
    at, bits, dt = _at(s["slots"], s["case"]["page_size"]), s["case"]["bits"], s["k_out"].dtype
    return [_values(s["k_cache"][at], s["k_scale"][at], bits).to(dt),
            _values(s["v_cache"][at], s["v_scale"][at], bits).to(dt)]


def _plain_attend(s):
    case = s["case"]
    size, bits, per = case["page_size"], case["bits"], case["per"]
    queries, heads, dim = s["q"].shape
    n, kv = queries // per, case["kv_heads"]
    table = s["table"].long().clamp(min=0)
    length = table.shape[1] * size

    def gathered(cache, pairs):  # [n][kv][length][dim]
        rows = cache[table].flatten(1, 2).transpose(1, 2)
        return _values(rows, pairs[table].flatten(1, 2).transpose(1, 2), bits)

    q = s["q"].float().reshape(n, per, kv, heads // kv, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = torch.matmul(q, gathered(s["k_cache"], s["k_scale"]).transpose(2, 3).contiguous())
    score = score.unflatten(2, (per, -1)) * s["scale"]
    live = torch.arange(length, device=table.device) < s["lens"].reshape(n, per)[..., None]
    score = score.masked_fill(~live[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), gathered(s["v_cache"], s["v_scale"]))
    out = out.unflatten(2, (per, -1)) / torch.where(total == 0, torch.ones_like(total), total)
    return out.permute(0, 2, 1, 3, 4).reshape(queries, heads, dim).to(s["q"].dtype)


# ---- the library's calls ----


def _calls(s):
    """The calls that a serving loop makes once for its buffers and keeps."""
    import prng_seeded_decode_amd as S

    op = s["case"]["op"]
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if op == "store":
        return [S.QCacheAppendCall(s["q"], s["k"], s["v"], s["cos"], s["sin"], s["positions"],
                                   s["slots"], s["q_out"], *cache,
                                   interleaved=s["case"]["interleaved"]),
                S.QCacheReadCall(*cache, s["slots"], s["k_back"], s["v_back"])]
    if op == "read":
        return [S.QCacheReadCall(*cache, s["slots"], s["k_out"], s["v_out"])]
    return [S.QCacheAttendCall(s["q"], *cache, s["table"], s["lens"], s["out"], scale=s["scale"],
                               rows=s["rows"])]


def _own(s):
    if "calls" not in s:
        s["calls"] = _calls(s)
    for call in s["calls"]:
        call()
    op = s["case"]["op"]
    if op == "store":
        return [s["q_out"], s["k_back"], s["v_back"], s["k_scale"], s["v_scale"]]
    if op == "read":
        return [s["k_out"], s["v_out"]]
    return s["out"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "store":
        return _plain_store(state)
    return _plain_read(state) if op == "read" else _plain_attend(state)


# ---- what a pass cannot do without ----


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    d, kv = case["dim"], case["kv_heads"]
    row = kv * (d * case["bits"] // 8 + 4 * (d // case["group"]))  # a token's keys in the cache
    if case["op"] == "store":
        # q in and out, k and v in, angles, codes and pairs out, what they stand for out
        moved = case["heads"] * d * 2 * e + 2 * kv * d * e + 8 + 4 * case["rot"] + 2 * row + 4 * kv * d
        return {"bytes": case["tokens"] * moved,
                "flops": case["tokens"] * (3 * case["rot"] * (case["heads"] + kv) + 12 * kv * d)}
    if case["op"] == "read":
        return {"bytes": case["tokens"] * (2 * row + 2 * kv * d * e + 4),
                "flops": case["tokens"] * 4 * kv * d}
    n, per = case["requests"], case["per"]
    tokens = (case["max_len"] + per) / 2 if case["ragged"] else case["max_len"]
    seen = max(tokens - per / 2, tokens / 2)  # of a query, on average
    return {"bytes": n * (tokens * (2 * row + 4 / case["page_size"])
                          + per * (2 * case["heads"] * d * e + 4)),
            "flops": 4 * n * per * seen * case["heads"] * d}


# ---- the definitions in 64 bits ----


def _turned(case, s, x):
    """A complex rotation of each pair, in 64 bits."""
    rot = case["rot"]
    turn = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"].long()][:, None, :]
    y = x.double().clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (
        slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _elements(cache, pairs, case):
    """Element by element of the rows [..., bytes], [..., groups, 2]: the values in 64 bits."""
    bits, dim = case["bits"], case["dim"]
    out = torch.empty((*cache.shape[:-1], dim), dtype=torch.float64, device=cache.device)
    for d in range(dim):
        bit = (d % 16) * (dim // 16 * bits) + d // 16 * bits
        code = (cache[..., bit // 8] >> (bit % 8)) & (2 ** bits - 1)
        pair = pairs[..., d // case["group"], :].double()
        out[..., d] = pair[..., 1] + pair[..., 0] * code
    return out


def _exact_store(case, s):
    size, group, top = case["page_size"], case["group"], 2 ** case["bits"] - 1
    keep = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][keep].long()
    at = (slot // size, slot % size)
    backs, pools = [], []
    for x, pool in ((_turned(case, s, s["k"]), s["k_scale"]), (s["v"].double(), s["v_scale"])):
        x = x.half().double()[keep].unflatten(-1, (-1, group))
        low, high = x.min(-1)[0], x.max(-1)[0]
        step = ((high - low) / top).half().double()
        code = ((x - low[..., None]) / step[..., None]).round().clamp(0, top)
        back = torch.zeros((case["tokens"], case["kv_heads"], case["dim"]), dtype=torch.float64,
                           device="cuda")
        back[keep] = (low[..., None] + step[..., None] * torch.nan_to_num(code)).flatten(-2)
        pool = pool.double().contiguous()
        pool[at] = torch.stack([step, low], -1)
        backs.append(back)
        pools.append(pool)
    return [_turned(case, s, s["q"]), *backs, *pools]


def _exact_read(case, s):
    slot, size = s["slots"].long(), case["page_size"]
    return [_elements(c[slot // size, slot % size], p[slot // size, slot % size], case)
            for c, p in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]))]


def _exact_attend(case, s):
    """Request by request over its own tokens."""
    size, per, kv, dim = case["page_size"], case["per"], case["kv_heads"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lens = s["lens"].reshape(-1, per)
    for b, length in enumerate(lens.amax(1).tolist()):
        if length == 0:
            continue
        pages = s["table"][b, : -(-length // size)].long()
        k, v = (_elements(c[pages].flatten(0, 1)[:length], p[pages].flatten(0, 1)[:length], case)
                for c, p in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
        hidden = torch.arange(length, device="cuda")[None, :] >= lens[b][:, None]
        for h in range(case["heads"]):
            g = h // (case["heads"] // kv)
            q = s["q"][b * per: (b + 1) * per, h].double()
            p = (q @ k[:, g].t().contiguous() * s["scale"]).masked_fill(hidden, -math.inf)
            out[b * per: (b + 1) * per, h] = torch.softmax(p, 1) @ v[:, g].contiguous()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    make = {"store": _exact_store, "read": _exact_read, "attend": _exact_attend}
    return make[case["op"]](case, s)
