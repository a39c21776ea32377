"""Infinities in an adapter's own operands: which outputs are infinite, and of which sign, and
which are NaN follows from the formula in 64 bits, whatever form the number of rows selects."""
import numpy as np
import pytest

import serve_ref as R
from test_gpu_lora import make, run

pytestmark = pytest.mark.gpu

# one launch, the row kernels, and the matrix cores with 16 and with 32 ranks a pass
FORMS = [(6, 16, (264, 512)), (96, 24, (264, 512)), (1030, 16, (2056, 2064)),
         (1400, 8, (4104, 2056)), (340, 64, (1032, 2056)), (129, 256, (1032, 1032))]


def check(c):
    import torch

    s = c["host"][0]
    for t, k in zip(c["dev"][0], ("x", "A", "B", "base")):
        t.copy_(torch.from_numpy(s[k]))
    got = run(c)[0]
    with np.errstate(invalid="ignore"):
        ref, tol = R.lora(*(s[k].astype(np.float64) for k in ("x", "A", "B", "base")), c["ids"],
                          c["scales"].astype(np.float64), c["y16"])
    for what in (np.isnan, np.isposinf, np.isneginf):
        assert (what(got) != what(ref)).sum() == 0, what
    fine = np.isfinite(ref)
    assert np.all(np.abs(got[fine] - ref[fine]) <= tol[fine])
    return ref


def case(tokens, rank, site, seed=31):
    return make([seed, tokens, rank], [site], rank, tokens, 4, np.arange(tokens) % 4)


@pytest.mark.parametrize("tokens,rank,site", FORMS)
def test_infinite_a_x(tokens, rank, site):
    # one rank of adapter 1 is infinite: every output takes the sign of its B, or is NaN where
    # that is 0; the other ranks' A x lie beyond fp16's range
    c = case(tokens, rank, site)
    s = c["host"][0]
    s["A"][1] = (s["A"][1].astype(np.float64) * 2.0 ** 12).astype(np.float16)
    s["x"][1::4] = (s["x"][1::4].astype(np.float64) * 2.0 ** 9).astype(np.float16)
    s["A"][1, 5, 7] = np.inf
    s["B"][1, 3, 5], s["B"][1, 200, 5] = 0, -0.0
    ref = check(c)
    assert np.isposinf(ref).any() and np.isneginf(ref).any() and np.isnan(ref[1, [3, 200]]).all()
    # x itself infinite, in one row
    c = case(tokens, rank, site)
    c["host"][0]["x"][2, 11] = -np.inf
    c["host"][0]["A"][2, :, 11] = np.abs(c["host"][0]["A"][2, :, 11]) + np.float16(0.1)
    c["host"][0]["B"][2, 17] = np.abs(c["host"][0]["B"][2, 17]) + np.float16(0.1)
    ref = check(c)
    assert np.isinf(ref[2, 17]) and np.isnan(ref[2]).any()


@pytest.mark.parametrize("tokens,rank,site", FORMS)
def test_infinite_b(tokens, rank, site):
    c = case(tokens, rank, site)
    s = c["host"][0]
    s["B"][2, 17, 5], s["B"][2, 101, 0], s["B"][2, 102, 7] = np.inf, -np.inf, -np.inf
    s["B"][2, 103, [2, 3]] = np.inf, -np.inf
    s["x"][2] = 0  # 0 times infinity
    ref = check(c)
    assert np.isnan(ref[2, 17]) and np.isinf(ref[[r for r in range(6, tokens, 4)], 17]).all()


@pytest.mark.parametrize("tokens,rank,site", FORMS)
def test_infinite_b_against_a_far_smaller_value_than_its_rows_largest(tokens, rank, site):
    # A x of rank 1 is 2^-40 of rank 0's
    c = case(tokens, rank, site)
    s = c["host"][0]
    s["x"][3::4] = 0
    s["x"][3::4, 9] = np.where(np.arange(len(s["x"][3::4])) % 2, 1.5, -2.0)
    s["A"][3, 0, 9], s["A"][3, 1, 9] = 49152.0, 2.0 ** -24
    s["B"][3, :, 0] = 2.0 ** -14
    s["B"][3, 40, 1], s["B"][3, 41, 1] = np.inf, -np.inf
    ref = check(c)
    assert np.isinf(ref[3::4, [40]]).all() and np.isinf(ref[3::4, [41]]).all()
