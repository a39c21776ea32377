"""Which adapter calls take the one-launch form, which alone needs no scratch (CPU only)."""
import ctypes

import pytest

import prng_seeded_decode_amd as S
from prng_seeded_decode_amd import _serve

P = 4096  # an aligned address that is never used


@pytest.mark.parametrize("rows,cols,rank,tokens,one", [
    (4096, 8192, 16, 16, True), (4096, 11008, 16, 16, True), (4096, 14336, 16, 1, True),
    (4096, 16384, 16, 32, True), (1024, 28672, 8, 4, True), (4096, 20480, 16, 4, False),
    (8192, 28672, 16, 1, False), (2048, 2048, 17, 1, False),
    (4096, 4096, 16, 256, True),
    (4096, 4096, 16, 257, False),
])
def test_one_launch_while_a_is_small_and_the_workgroups_fit(rows, cols, rank, tokens, one):
    site = (_serve._LoraSite * 1)(_serve._LoraSite(P, P, P, P, P, rows, cols, rank))
    n = ctypes.c_size_t(0)
    assert S.lib().seedlm_lora_scratch_bytes(ctypes.cast(site, ctypes.c_void_p), 1, tokens, 4, S.F16,
                                             S.F16, ctypes.byref(n)) == S.OK
    assert (n.value == 0) == one
