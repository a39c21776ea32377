"""Plain 64-bit forms of the serving operators for the tests, and the bounds that go with them.

u32 and u16 are the half-steps of fp32 and fp16 relative to a value (2^-24, 2^-11); fp16 values
below 2^-14 lie 2^-24 apart.  A sum of products whose additions form a tree of depth n is off by
at most n * u32 times the sum of the products' magnitudes (first order)."""
import numpy as np

U32, U16 = 2.0 ** -24, 2.0 ** -11


def rounding(ref, f16):
    """Half a step of the output's type at ref."""
    return np.abs(ref) * U16 + 2.0 ** -25 if f16 else np.abs(ref) * U32


def plan(lens, fresh, table, ring, ring_state, page_size, tokens):
    """Request by request, page by page; returns all nine outputs."""
    table, ring = np.array(table, np.int64), [int(v) for v in ring]
    head, count = int(ring_state[0]), int(ring_state[1])
    n, most = table.shape
    pool = len(ring)
    ring_out, lens_out = list(ring), [int(v) for v in lens]
    offsets, ok = [0], []
    rows, positions, slots = [-1] * tokens, [0] * tokens, [-1] * tokens
    wanted = popped = pushed = 0
    for b in range(n):
        length, new = int(lens[b]), max(int(fresh[b]), 0)
        start = offsets[-1]
        offsets.append(start + new)
        held = -(-length // page_size)
        granted = True
        if fresh[b] < 0:
            for j in range(held):
                ring_out[(head + count + pushed) % pool] = int(table[b, j])
                pushed += 1
            lens_out[b] = 0
        elif length + new > most * page_size or start + new > tokens:
            granted = False
        else:
            need = -(-(length + new) // page_size) - held
            wanted += need
            if need > 0 and wanted > count:
                granted = False
            else:
                for j in range(need):
                    table[b, held + j] = ring[(head + popped + j) % pool]
                popped += need
                lens_out[b] = length + new
        ok.append(int(granted))
        for i in range(start, min(start + new, tokens)):
            rows[i], positions[i] = b, length + i - start
            if granted:
                page = int(table[b, positions[i] // page_size])
                if 0 <= page < pool:
                    slots[i] = page * page_size + positions[i] % page_size
    return dict(lens_out=lens_out, ring_state_out=[(head + popped) % pool, count - popped + pushed],
                offsets=offsets, rows=rows, positions=positions, slots=slots, ok=ok,
                table=table.tolist(), ring=ring_out)


def rotate(x, cos, sin, interleaved):
    """x [tokens][heads][dim], cos and sin [tokens][rot/2]: the rotation and its error bound
    (two products and a sum in fp32)."""
    y, off = x.astype(np.float64).copy(), np.zeros(x.shape)
    half = cos.shape[1]
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = y[..., first].copy(), y[..., second].copy()
    c, s = cos.astype(np.float64)[:, None, :], sin.astype(np.float64)[:, None, :]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    off[..., first] = 2 * U32 * (np.abs(a * c) + np.abs(b * s))
    off[..., second] = 2 * U32 * (np.abs(b * c) + np.abs(a * s))
    return y, off


def attend(q, keys, values, scale, f16):
    """One request: q [heads][dim], keys and values [tokens][kv_heads][dim] (float64).  Returns
    the output and its error bound, element by element."""
    heads, dim = q.shape
    n, kv = keys.shape[:2]
    out, tol = np.zeros((heads, dim)), np.zeros((heads, dim))
    if n == 0:
        return out, tol
    for h in range(heads):
        k, v = keys[:, h // (heads // kv)], values[:, h // (heads // kv)]
        s = k @ q[h] * scale
        p = np.exp(s - s.max())
        w = p / p.sum()
        out[h] = w @ v
        # A score: dim products in fp32 sums, fp32 queries to 2^-22 of the row's largest, the
        # scale's two roundings and the subtraction of the maximum.
        es = (np.abs(k) @ np.abs(q[h]) * abs(scale)).max() * (dim + 4) * U32
        es += np.abs(k).sum(1).max() * np.abs(q[h]).max() * abs(scale) * 2.0 ** -22
        es += 4 * U32 * np.abs(s).max()
        # A weight: its score's and the maximum's errors, exp2 (2 units), 22 bits in two parts.
        # Sums: 32 tokens of a tile, two parts, n/128 tiles, 4 waves, the join of at most n/128
        # pieces; numerator and denominator.
        weight = 2 * es + 4 * U32 + 2.0 ** -21
        depth = 2 * (32 + 2 * (n / 128 + 1) + 8 + n / 128 + 1)
        tol[h] = 2 * (weight + depth * U32) * (w @ np.abs(v))
    return out, tol + rounding(out, f16)


def lora(x, A, B, base, adapter, scales, f16):
    """y and its bound: float64 inputs, x [tokens][cols], A [n][rank][cols], B [n][rows][rank]."""
    y = base.copy()
    tol = np.zeros(base.shape)
    rank, cols = A.shape[1:]
    for a in range(A.shape[0]):
        at = np.nonzero(adapter == a)[0]
        if at.size == 0:
            continue
        h = x[at] @ A[a].T
        y[at] += scales[a] * (h @ B[a].T)
        # A x: sums of cols products (no deeper than cols / 8 + 64); the second product: rank
        # of them, A x in 22 bits of its row's largest, the scale, and the addition of base.
        eh = (cols / 8 + 64) * U32 * (np.abs(x[at]) @ np.abs(A[a]).T)
        eh += 2.0 ** -21 * np.abs(h).max(1, keepdims=True)
        tol[at] = abs(scales[a]) * ((eh + (rank + 8) * U32 * np.abs(h)) @ np.abs(B[a]).T)
        tol[at] += 2 * U32 * np.abs(y[at])
    return y, tol + rounding(y, f16)
