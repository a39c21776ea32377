"""seedlm_qcache_attend in calls whose tables may hold more codes than the caches are taken to
(110 MB), which read codes past them: the forms of 64 dimensions and of one group of 256, and calls
that are not split."""
import numpy as np
import pytest

from test_gpu_qcache_attend import check, make, run, widen

pytestmark = pytest.mark.gpu


def held(x, cap):
    """Bytes that a call of these requests may read, by its sizes."""
    pages, size, kv, width = x["cache"][0].shape
    return len(x["lens"]) * cap * kv * 2 * (width + 4 * x["cache"][2].shape[3])


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("heads,kv,dim,bits,groups,size,head_major", [
    (8, 2, 64, 8, 1, 16, False), (20, 1, 64, 8, 2, 7, True), (5, 5, 64, 8, 1, 48, True),
    (4, 2, 256, 4, 1, 16, True), (18, 1, 256, 4, 1, 100, False)])
def test_split_calls(heads, kv, dim, bits, groups, size, head_major, f16):
    lens = [0, 1, 33, 128, 129, 700, 3000, 255, 2049, 0]
    x = make([heads, dim, size, 9], lens, heads, kv, dim, size, f16, bits, groups, head_major)
    x = widen(x, (2 ** 28 // held(x, 1)) // size + 1, wild=-(2 ** 31))
    assert held(x, x["dtable"].shape[1] * size) > 2 ** 27
    check(x, run(x))


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dim,bits,groups,cap", [
    (64, 8, 1, 2048), (64, 8, 2, 2048), (128, 4, 1, 2048), (128, 8, 4, 2048), (256, 4, 1, 1024),
    (256, 4, 4, 1024)])
def test_whole_calls(dim, bits, groups, cap, f16):
    import torch

    import prng_seeded_decode_amd as S

    rng = np.random.default_rng(dim + groups)
    lens = np.minimum(np.exp(rng.uniform(0, np.log(300), 300)).astype(int) * rng.integers(0, 2, 300), 290)
    lens[7] = cap
    x = widen(make([dim, groups, 3], [int(v) for v in lens], 8, 2, dim, 16, f16, bits, groups), cap // 16)
    assert held(x, cap) > 2 ** 27
    call = S.QCacheAttendCall(x["dq"], *x["cache"], x["dtable"], x["dlens"], torch.empty_like(x["dq"]))
    assert call.scratch_bytes() == 0
    check(x, run(x))
