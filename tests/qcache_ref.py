"""A quantised cache for the tests: its layout written out element by element, its quantisation
in the fp32 steps that define it, and attention over it in 64 bits with error bounds."""
import numpy as np

import serve_ref as R
from serve_ref import U32


def places(dim, bits):
    """Byte and shift of each element of a row: unit d % 16, place d // 16 in it."""
    at = [(d % 16) * (dim // 16) + d // 16 for d in range(dim)]
    return [(p * bits // 8, p * bits % 8) for p in at]


def pack(codes, bits):
    """Codes [..., dim] as rows of bytes."""
    dim = codes.shape[-1]
    rows = np.zeros((*codes.shape[:-1], dim * bits // 8), np.uint8)
    for d, (byte, shift) in enumerate(places(dim, bits)):
        rows[..., byte] |= (codes[..., d].astype(np.uint32) << shift).astype(np.uint8)
    return rows


def unpack(rows, bits):
    dim = rows.shape[-1] * 8 // bits
    out = np.zeros((*rows.shape[:-1], dim), np.int64)
    for d, (byte, shift) in enumerate(places(dim, bits)):
        out[..., d] = (rows[..., byte] >> shift) & (2 ** bits - 1)
    return out


def values(rows, pairs, bits):
    """What rows [..., bytes] with pairs [..., groups, 2] stand for, and the magnitude of its two
    terms, in 64 bits."""
    c = unpack(rows, bits).astype(np.float64)
    groups = pairs.shape[-2]
    c = c.reshape(*c.shape[:-1], groups, -1)
    p = pairs.astype(np.float64)
    with np.errstate(invalid="ignore"):
        scaled, offset = p[..., :1] * c, p[..., 1:]
        shape = (*rows.shape[:-1], -1)
        return (offset + scaled).reshape(shape), (np.abs(offset) + np.abs(scaled)).reshape(shape)


def rotate32(x, cos, sin, interleaved):
    """The rotation of x [tokens][heads][dim] in fp32, each operation rounded, then fp16."""
    y = x.astype(np.float32).copy()
    half = cos.shape[1]
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = y[..., first].copy(), y[..., second].copy()
    c, s = cos[:, None, :], sin[:, None, :]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    with np.errstate(over="ignore"):
        return y.astype(np.float16)


def quantise(x, bits, group):
    """Rows of bytes and pairs of fp16 values x [..., dim], by the definition's steps."""
    levels = np.float32(2 ** bits - 1)
    g = x.astype(np.float32).reshape(*x.shape[:-1], -1, group)
    finite = np.isfinite(g).all(-1)
    g = np.where(finite[..., None], g, np.float32(0))
    low, high = g.min(-1), g.max(-1)
    scale = ((high - low) / levels).astype(np.float16)
    s = scale.astype(np.float32)[..., None]
    code = np.rint((g - low[..., None]) / np.where(s == 0, np.float32(1), s))
    code = np.where(s == 0, 0, np.minimum(code, levels)).astype(np.int64)
    scale = np.where(finite, scale, np.float16(np.nan))
    offset = np.where(finite, low, 0).astype(np.float16)
    return pack(code.reshape(x.shape), bits), np.stack([scale, offset], -1)


def attend(q, k, kmag, v, vmag, scale, f16):
    """One query: q [heads][dim], k, v and the magnitudes of their terms [tokens][kv_heads][dim].
    Returns the output and its error bound, element by element."""
    heads, dim = q.shape
    n, kv = k.shape[:2]
    out, tol = np.zeros((heads, dim)), np.zeros((heads, dim))
    if n == 0:
        return out, tol
    for h in range(heads):
        j = h // (heads // kv)
        s = k[:, j] @ q[h] * scale
        p = np.exp(s - s.max())
        w = p / p.sum()
        out[h] = w @ v[:, j]
        # A score: fp32 sums of dim products of codes and of dim offsets, a product and a sum for
        # each of up to 4 groups (offset and code terms may cancel, so their magnitudes count),
        # queries to 2^-22 of the row's largest, the scale's roundings, the maximum's subtraction.
        es = (kmag[:, j] @ np.abs(q[h]) * abs(scale)).max() * (dim + 16) * U32
        es += kmag[:, j].sum(1).max() * np.abs(q[h]).max() * abs(scale) * 2.0 ** -22
        es += 4 * U32 * np.abs(s).max()
        # A weight: its score's and the maximum's errors, exp2 (2 units), the product with the
        # value's scale, 22 bits in two parts.  Sums: 32 tokens of a tile, two parts, n/128 tiles,
        # 4 waves, the join of at most n/128 pieces; numerator and denominator, the latter's
        # offset part too.
        weight = 2 * es + 6 * U32 + 2.0 ** -21
        depth = 2 * (32 + 2 * (n / 128 + 1) + 8 + n / 128 + 1)
        tol[h] = 2 * (weight + depth * U32) * (w @ vmag[:, j])
    return out, tol + R.rounding(out, f16)
