"""seedlm_lora_many against the sums in 64 bits, element by element within serve_ref.lora's
bounds."""
import numpy as np
import pytest

import serve_ref as R

pytestmark = pytest.mark.gpu


def make(seed, sites, rank, tokens, adapters, ids, x16=True, y16=True, offset=0):
    """offset: elements by which every tensor starts past an aligned address."""
    import torch

    rng = np.random.default_rng(seed)
    tens = []

    def dev(a):
        flat = torch.zeros(a.size + offset, dtype=torch.from_numpy(a).dtype, device="cuda")
        t = flat[offset:].view(a.shape)
        t.copy_(torch.from_numpy(a))
        return t

    host = []
    for rows, cols in sites:
        s = {"x": rng.standard_normal((tokens, cols)).astype(np.float16 if x16 else np.float32),
             "A": (rng.standard_normal((adapters, rank, cols)) * cols ** -0.5).astype(np.float16),
             "B": (rng.standard_normal((adapters, rows, rank)) * rank ** -0.5).astype(np.float16),
             "base": rng.standard_normal((tokens, rows)).astype(np.float16 if y16 else np.float32)}
        host.append(s)
        tens.append([dev(s[k]) for k in ("x", "A", "B", "base")])
    scales = rng.uniform(-2, 2, adapters).astype(np.float32)
    return {"host": host, "dev": tens, "ids": np.asarray(ids), "scales": scales,
            "dids": torch.from_numpy(np.asarray(ids, np.int32)).cuda(),
            "dscales": torch.from_numpy(scales).cuda(), "y16": y16}


def run(c, in_place=False, stream=None):
    import torch

    import prng_seeded_decode_amd as S

    sites = []
    for x, A, B, base in c["dev"]:
        base = base.clone() if in_place else base
        y = base if in_place else torch.full_like(base, 9.0)
        sites.append((x, A, B, base, y))
    torch.cuda.synchronize()
    ys = S.seedlm_lora_many(sites, c["dids"], c["dscales"], stream=stream)
    torch.cuda.synchronize()
    return [y.double().cpu().numpy() for y in ys]


def check(c, got):
    for s, y in zip(c["host"], got):
        ref, tol = R.lora(*(s[k].astype(np.float64) for k in ("x", "A", "B", "base")), c["ids"],
                          c["scales"].astype(np.float64), c["y16"])
        none = (c["ids"] < 0) | (c["ids"] >= len(c["scales"]))
        assert np.array_equal(y[none], s["base"].astype(np.float64)[none])
        err = np.abs(y - ref)
        assert np.all(err <= tol), (float((err - tol).max()), float(err.max()))


def ids_of(seed, tokens, adapters, kind):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full(tokens, adapters - 1)
    if kind == "none":
        return rng.choice([-1, adapters, 2 ** 31 - 1, -2 ** 31], tokens)
    if kind == "mixed":
        return rng.integers(-1, adapters + 1, tokens)
    cuts = np.sort(rng.integers(0, tokens + 1, min(tokens, 7)))  # requests, one after another
    return rng.integers(-1, adapters, len(cuts) + 1)[np.searchsorted(cuts, np.arange(tokens), "right")]


@pytest.mark.parametrize("x16,y16", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("tokens,rank,sites", [
    (1, 16, [(256, 512)]), (1, 8, [(2048, 2048)]), (3, 16, [(512, 1032), (128, 1032)]),
    (16, 64, [(1000, 776)]), (5, 5, [(33, 47)]), (7, 1, [(1, 1)]), (2, 256, [(300, 264)]),
    (4, 24, [(264, 96), (8, 3000), (520, 88)]), (16, 12, [(65, 2050)]),
])
@pytest.mark.parametrize("kind", ["mixed", "one"])
def test_lora_of_few_rows(tokens, rank, sites, kind, x16, y16):
    c = make([tokens, rank], sites, rank, tokens, 6, ids_of([tokens], tokens, 6, kind), x16, y16)
    check(c, run(c))
    check(c, run(c, in_place=True))


@pytest.mark.parametrize("kind", ["requests", "mixed", "one", "none"])
@pytest.mark.parametrize("tokens,rank,sites", [
    (17, 16, [(512, 256)]), (33, 8, [(264, 520), (128, 520)]), (64, 32, [(1000, 776)]),
    (129, 64, [(72, 1096)]), (200, 16, [(1024, 1024), (256, 1024), (256, 1024)]),
    (77, 24, [(520, 264)]), (130, 128, [(136, 264)]), (50, 256, [(200, 136)]),
    (40, 5, [(33, 47)]), (65, 20, [(130, 100)]), (35, 16, [(8, 8)]), (257, 48, [(328, 2056)]),
    # enough products for the matrix cores (128 MiB of A and B, counted once per row)
    (1030, 16, [(2056, 2064)]), (129, 256, [(1032, 1032)]), (300, 64, [(1800, 1720)]),
    (700, 24, [(2056, 1944)]), (1030, 8, [(4104, 2056), (264, 2056)]), (400, 128, [(680, 680)]),
    (4200, 16, [(1000, 1000)]), (64, 240, [(3208, 1200)]), (700, 32, [(8, 3000)]),
])
def test_lora_of_many_rows(tokens, rank, sites, kind):
    c = make([tokens, rank, 1], sites, rank, tokens, 5, ids_of([tokens], tokens, 5, kind))
    check(c, run(c))
    check(c, run(c, in_place=True))


def test_lora_of_many_fp32_rows_and_of_unaligned_tensors():
    c = make([21], [(264, 520)], 16, 70, 4, ids_of([1], 70, 4, "mixed"), False, False)
    check(c, run(c))
    for tokens in (3, 70):
        c = make([22], [(264, 520)], 16, tokens, 4, ids_of([1], tokens, 4, "mixed"), offset=1)
        check(c, run(c))


def test_lora_of_more_sites_than_one_launch_takes():
    sites = [(64 + 8 * i, 128 + 8 * i) for i in range(19)]
    for tokens in (2, 40):
        c = make([23], sites, 8, tokens, 3, ids_of([2], tokens, 3, "mixed"))
        check(c, run(c))


# one launch, the row kernels, the matrix cores
FORMS = [(6, 16, (264, 512)), (96, 24, (264, 512)), (340, 64, (1032, 2056))]


@pytest.mark.parametrize("tokens,rank,site", FORMS)
def test_lora_keeps_other_adapters_nan_and_infinities_away(tokens, rank, site):
    c = make([24], [site], rank, tokens, 4, np.arange(tokens) % 4)
    clean = run(c)[0]
    x, A, B, base = c["dev"][0]
    A[1, 3, 100], B[2, 17, 5], x[3, 9] = float("nan"), float("inf"), float("nan")
    got = run(c)[0]
    own = np.arange(tokens) % 4
    assert np.isnan(got[own == 1]).all()
    assert np.array_equal(got[own == 0], clean[own == 0])
    assert np.array_equal(np.delete(got[own == 2], 17, 1), np.delete(clean[own == 2], 17, 1))
    assert not np.isfinite(got[own == 2][:, 17]).any()
    rest = (own == 3) & (np.arange(tokens) != 3)
    assert np.array_equal(got[rest], clean[rest]) and np.isnan(got[3]).all()


@pytest.mark.parametrize("y16", [True, False])
@pytest.mark.parametrize("tokens,rank,site", FORMS)
def test_lora_of_large_and_small_products(tokens, rank, site, y16):
    # A x beyond fp16's range, and far below its normal numbers
    for power in (9, -20):
        c = make([25], [site], rank, tokens, 3, np.arange(tokens) % 3, True, y16)
        s = c["host"][0]
        s["x"] = (s["x"].astype(np.float64) * 2.0 ** power).astype(np.float16)
        s["A"] = (s["A"].astype(np.float64) * (2.0 ** 9 if power > 0 else 1)).astype(np.float16)
        if power > 0:
            s["B"] = (s["B"].astype(np.float64) * 2.0 ** -14).astype(np.float16)
        import torch

        for i, k in enumerate(("x", "A", "B")):
            c["dev"][0][i].copy_(torch.from_numpy(s[k]))
        check(c, run(c))


@pytest.mark.parametrize("tokens,rank,site", FORMS)
def test_lora_on_another_stream_and_in_a_graph(tokens, rank, site):
    import torch

    import prng_seeded_decode_amd as S

    c = make([26], [site, (128, site[1])], rank, tokens, 4, ids_of([3], tokens, 4, "mixed"))
    plain = run(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert all(np.array_equal(a, b) for a, b in zip(run(c, stream=side), plain))
    sites = [(x, A, B, base, torch.zeros_like(base)) for x, A, B, base in c["dev"]]
    call = S.LoraCall(sites, c["dids"], c["dscales"])
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for seed in range(4):
        ids = ids_of([seed, 9], tokens, 4, "mixed")
        c["dids"].copy_(torch.from_numpy(ids.astype(np.int32)))
        c["ids"] = ids
        graph.replay()
        torch.cuda.synchronize()
        got = [s[4].double().cpu().numpy() for s in sites]
        check(c, got)
        assert all(np.array_equal(a, b) for a, b in zip(run(c), got))


def test_lora_beside_a_packed_projection():
    """base from seedlm_gemv: the packed weights and the adapter together, against 64 bits of
    the decoded weights; the projection's own fp16 tolerance comes on top."""
    import torch

    import prng_seeded_decode_amd as S
    from workloads import gen_records

    rows, cols, n = 256, 512, 3
    m = S.seedlm_pack(*gen_records(9, 1, rows, cols, 8, 3), rows, cols, 8, 3, 16)
    c = make([27], [(rows, cols)], 16, n, 2, [0, -1, 1])
    W = torch.empty((rows, cols), dtype=torch.float32, device="cuda")
    S.seedlm_decode(m, W)
    x, A, B, base = c["dev"][0]
    S.seedlm_gemv(m, x, base, batch=n)
    S.seedlm_lora_many([(x, A, B, base, base)], c["dids"], c["dscales"])
    torch.cuda.synchronize()
    s = c["host"][0]
    s["base"] = (s["x"].astype(np.float64) @ W.double().cpu().numpy().T)
    ref, _ = R.lora(*(s[k].astype(np.float64) for k in ("x", "A", "B", "base")), c["ids"],
                    c["scales"].astype(np.float64), True)
    got = base.double().cpu().numpy()
    assert np.linalg.norm(got - ref) <= 2e-3 * np.linalg.norm(ref)
    m.destroy()


@pytest.mark.parametrize("adapters,tokens,rank,site", [
    (300, 2100, 16, (1000, 1048)), (8191, 16100, 8, (520, 8)), (8200, 16100, 8, (520, 8))])
def test_lora_of_many_adapters(adapters, tokens, rank, site):
    # tiles of a row or two each, and more adapters than the sort takes
    rng = np.random.default_rng(adapters)
    ids = rng.integers(-1, adapters + 1, tokens)
    ids[: tokens // 3] = 7
    c = make([28, adapters], [site], rank, tokens, adapters, ids)
    check(c, run(c))
    check(c, run(c, in_place=True))
