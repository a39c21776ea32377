"""seedlm_qcache_attend where numbers lie far apart: scores whose steps in fp32 are whole powers of
two, and values' scales that differ from token to token and from group to group by more than the
bits of a softmax weight.  Offsets of values are 0 here, so that nothing hides what codes and
scales give; bounds are those of qcache_ref.attend and what is said beside each."""
import numpy as np
import pytest

import qcache_ref as Q
from test_gpu_qcache_attend import check, make, run, run_rows, terms, widen

pytestmark = pytest.mark.gpu

FORMS = [(64, 4, 1), (64, 8, 2), (128, 4, 1), (128, 8, 4), (128, 4, 2), (256, 4, 4), (256, 8, 1)]


def values_of(x, b, scale, offset=0.0):
    """Gives request b's values the scales `scale` ([tokens], [tokens][1][groups] or a number)."""
    import torch

    p, t = np.array(x["where"][b]).T
    s = np.zeros(tuple(x["cache"][3][p, t].shape[:-1]))
    s[:] = scale[:, None, None] if np.ndim(scale) == 1 else scale
    pairs = np.stack([s, np.full_like(s, offset)], -1).astype(np.float16)
    assert np.isfinite(pairs).all()
    x["cache"][3][p, t] = torch.from_numpy(pairs).cuda()
    x["terms"][b] = terms(x, b)


def keys_of(x, b, tokens, offset):
    """Makes every element of the keys of request b's `tokens` (None: all) `offset`, a number or
    one for each token."""
    import torch

    p, t = np.array(x["where"][b])[slice(None) if tokens is None else tokens].T
    pairs = np.zeros(tuple(x["cache"][2][p, t].shape), np.float16)
    pairs[..., 1] = np.reshape(offset, (-1, 1, 1))
    x["cache"][2][p, t] = torch.from_numpy(pairs).cuda()
    x["terms"][b] = terms(x, b)


def uneven(n, dim):
    """Keys that give n tokens scores of -1 to 0 by a query of ones: weights of all their bits."""
    return -np.random.default_rng(n).uniform(0, 1, n) / dim


def ones(x, value=1.0):
    import torch

    x["q"][:] = value
    x["dq"] = torch.from_numpy(x["q"]).cuda()


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dim,bits,groups", FORMS)
@pytest.mark.parametrize("key,query", [(2000.0, 2000.0), (60000.0, 60000.0), (-500.0, 3000.0)])
def test_scores_past_24_bits(key, query, dim, bits, groups, f16):
    # All scores of a request are one number, of 2^26 to 2^40 in powers of 2, where fp32's steps are
    # 4 to 2^17: weights of one another's size all the same, whole and split.  The mean of the
    # values, exact in the scores, so that the bound is that of scores of 0.
    lens = [700, 40, 1, 129]
    x = make([dim, bits, 31], lens, 4, 2, dim, 16, f16, bits, groups)
    for b in range(4):
        values_of(x, b, 0.25 if bits == 4 else 0.02)
        keys_of(x, b, None, 0.0)
    ones(x, query)
    want = [[a.copy() for a in t] for t in x["terms"]]
    for b in range(4):
        keys_of(x, b, None, key)
    x["terms"] = want
    for y in (x, widen(x, 1024)):
        check(y, run(y, scale=1.0), scale=1.0)


@pytest.mark.parametrize("f16", [True, False])
def test_the_largest_of_scores_past_24_bits_takes_all(f16):
    # One token above the others by far more than a step, in each of three tiles and waves.
    for at in (3, 70, 699):
        x = make([at, 32], [700], 4, 2, 128, 16, f16, 4, 1)
        values_of(x, 0, 0.5)
        keys_of(x, 0, None, 1900.0)
        keys_of(x, 0, [at], 2000.0)
        ones(x, 2000.0)
        _, _, v, _ = x["terms"][0]
        for y in (x, widen(x, 1024)):
            got = run(y, scale=1.0)
            assert np.array_equal(got[0], np.repeat(v[at], 2, 0))  # multiples of 1/2 below 8


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dim,bits,groups", FORMS)
@pytest.mark.parametrize("power", [0, -10, -17, -24])
def test_a_large_scale_of_no_weight_costs_the_others_nothing(power, dim, bits, groups, f16):
    # Token 5, of scale 2^12, has at most e^-63 of another's weight, so 2^-54 of its term: the
    # reference is without it.
    lens = [700, 130]
    x = make([dim, bits, 33], lens, 4, 2, dim, 16, f16, bits, groups)
    for b, n in enumerate(lens):
        s = np.full(n, 2.0 ** power)
        s[5] = 2.0 ** 12
        values_of(x, b, s)
        keys_of(x, b, None, uneven(n, dim))
        keys_of(x, b, [5], -64.0 / dim)
        x["terms"][b] = [np.delete(a, 5, 0) for a in x["terms"][b]]
    ones(x)
    for y in (x, widen(x, 1024)):
        check(y, run(y, scale=1.0), scale=1.0, lens=[n - 1 for n in lens])


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dim,bits,groups", [f for f in FORMS if f[2] > 1])
def test_groups_of_scales_far_apart(dim, bits, groups, f16):
    # Each group's elements are bounded by that group's own magnitudes.  Scores are 0 in the first
    # request, which leaves the weights' bits alone.
    lens = [700, 130, 1]
    for powers in ([12, -20, -24, 3], [-24, 12, 0, -10], [-10, 2, 11, -3], [-20, -24, -15, -17]):
        x = make([dim, bits, 34], lens, 4, 2, dim, 16, f16, bits, groups)
        for b, n in enumerate(lens):
            rng = np.random.default_rng(b)
            s = 2.0 ** np.array(powers[:groups]) * np.exp2(rng.uniform(0, 0.9, (n, 1, groups)))
            values_of(x, b, s)
        keys_of(x, 0, None, 0.0)
        for y in (x, widen(x, 1024)):
            check(y, run(y))


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dim,bits,groups", FORMS)
def test_elements_that_large_scales_leave_out(dim, bits, groups, f16):
    # 128 tokens of scale 2^12 whose codes are 0 in the last half of the elements, before, between
    # and after tokens of scale 2^-17: those elements keep the bits of the small scales.
    lens = [700]
    for first in (0, 256, 512):
        x = make([dim, bits, 35], lens, 4, 2, dim, 16, f16, bits, groups)
        s = np.full(700, 2.0 ** -17)
        s[first: first + 128] = 2.0 ** 12
        p, t = np.array(x["where"][0])[first: first + 128].T
        rows = x["cache"][1][p, t].unflatten(-1, (16, -1))
        rows[..., rows.shape[-1] // 2:] = 0
        x["cache"][1][p, t] = rows.flatten(-2)
        values_of(x, 0, s)
        keys_of(x, 0, None, uneven(700, dim))
        ones(x)
        for y in (x, widen(x, 1024)):
            check(y, run(y, scale=1.0), scale=1.0)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dim,bits,groups", [f for f in FORMS if f[2] > 1])
def test_a_group_that_the_heaviest_token_leaves_out(dim, bits, groups, f16):
    # Token 7 has e^10 of the others' weights, a scale of 0 in the first group, where the others have
    # 2^-20, and theirs in the rest.
    x = make([dim, bits, 36], [700], 4, 2, dim, 16, f16, bits, groups)
    s = np.ones((700, 1, groups))
    s[:, :, 0], s[7, :, 0] = 2.0 ** -20, 0.0
    values_of(x, 0, s)
    keys = uneven(700, dim)
    keys[7] = 10.0 / dim
    keys_of(x, 0, None, keys)
    ones(x)
    for y in (x, widen(x, 1024)):
        check(y, run(y, scale=1.0), scale=1.0)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("heads,kv", [(4, 2), (16, 2), (5, 1)])
@pytest.mark.parametrize("dim,bits,groups", [(128, 4, 2), (64, 8, 1), (256, 4, 4)])
def test_scales_past_one_querys_length_leave_its_bits(dim, bits, groups, heads, kv, f16):
    # Queries that share their reading: finite scales that only the longer ones attend to, behind
    # other tiles and in the first.
    import torch

    for n, at, lens in ((400, 380, [100, 400, 390, 380, 10, 381]), (30, 5, [5, 30, 6, 1, 4, 5])):
        x = make([16, heads, n], [n], heads, kv, dim, 16, f16, bits, groups)
        g = torch.Generator(device="cuda").manual_seed(n)
        q = torch.randn((6, heads, dim), generator=g, device="cuda").to(x["dq"].dtype)
        host, rows = q.cpu().numpy(), [0] * 6
        s = np.full(n, 2.0 ** -12)
        values_of(x, 0, s)
        clean = [run_rows(y, q, rows, lens) for y in (x, widen(x, 9000))]
        s[at:] = 2.0 ** 12
        values_of(x, 0, s)
        short = [i for i in range(6) if lens[i] <= at]
        for y, was in zip((x, widen(x, 9000)), clean):
            got = run_rows(y, q, rows, lens)
            for i in short:
                assert np.array_equal(got[i], was[i]), i
            check(y, got[short], lens=[lens[i] for i in short], rows=[0] * len(short), q=host[short])
            for i in set(range(6)) - set(short):
                ref, tol = Q.attend(host[i].astype(np.float64), *(a[: lens[i]] for a in y["terms"][0]),
                                    np.float64(np.float32(dim ** -0.5)), f16)
                # 32 tokens of which some have these scales: weights times scales, 2^15 standing for
                # the largest weight times 2^15 or less, are cut to 2^-24, so to 2^-24 of it, and the
                # products' sum to that many times the codes.
                tol += 2.0 ** -24 * np.repeat((x["terms"][0][3] / s[:, None, None])[at // 32 * 32:][:32].sum(0),
                                              heads // kv, 0)
                err = np.abs(got[i] - ref)
                if f16:
                    err[(np.abs(ref) + tol >= 65520) & (got[i] == np.copysign(np.inf, ref))] = 0
                assert np.all(err <= tol), (i, float((err - tol).max()))


@pytest.mark.parametrize("dim,bits,groups", FORMS)
def test_weights_are_not_low_on_average(dim, bits, groups):
    # Requests of one token with scores of any fraction, fp32: an output is its value times the
    # ratio of the weight's two parts to the weight.  Each ratio errs by at most 2^-22, half a step
    # of the second part, and with the roundings of a product, the join and the division by no more
    # than 2^-21; nearest roundings are as often high as low, so the mean over 512 columns lies
    # within 2^-21 / sqrt(512) < 2^-25.  (Parts that are cut leave 7.5e-8, more than 2^-24.)
    x = make([dim, groups, 5], [1] * 64, 8, 2, dim, 16, False, bits, groups)
    for b in range(64):
        values_of(x, b, 1.0)
    got = run(x)
    value = np.stack([np.repeat(x["terms"][b][2][0], 4, 0) for b in range(64)])
    with np.errstate(divide="ignore", invalid="ignore"):
        error = np.where(value > 0, got / value - 1, 0.0).sum(2) / (value > 0).sum(2)
    assert np.abs(error).max() <= 2.0 ** -21
    assert abs(error.mean()) < 2.0 ** -25, error.mean()


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dim,bits,groups", [f for f in FORMS if f[2] > 1])
@pytest.mark.parametrize("pair", [(np.nan, 0), (np.inf, 0), (1, np.inf), (1, -np.inf)])
def test_pairs_that_are_not_finite_beside_scales_far_apart(pair, dim, bits, groups, f16):
    # a token's first group is not finite; its last has a scale far above all others', or below
    import torch

    lens = [200, 33, 1, 700]
    x = make([dim, groups, 6], lens, 8, 2, dim, 16, f16, bits, groups)
    tokens = [(0, 150), (1, 32), (2, 0), (3, 1), (3, 600)]
    for power in (10, -10):
        for b, n in enumerate(lens):
            s = np.full((n, 2, groups), 2.0 ** -4)
            for r, t in tokens:
                if r == b:
                    s[t, :, -1] = 2.0 ** power
            values_of(x, b, s)
        clean = [run(y) for y in (x, widen(x, 9000))]
        for r, t in tokens:
            page, row = x["where"][r][t]
            x["cache"][3][page, row, :, 0] = torch.tensor(pair, dtype=torch.float16)
        for y, was in zip((x, widen(x, 9000)), clean):
            check(y, was)
            got = run(y)
            assert not np.isfinite(got[..., : dim // groups]).any()
            got[..., : dim // groups] = was[..., : dim // groups]
            check(y, got)
