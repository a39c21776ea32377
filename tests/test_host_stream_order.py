"""The launches that calls make (CPU only): host_stream_order_check.cpp loads the built library on
top of a stand-in for the HIP runtime and looks at their order, where several host threads call on
one stream, and at the kernel that a call's sizes select."""
import os
import subprocess

import pytest

from prng_seeded_decode_amd import _binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not available")
    _binding.lib()  # it has been built
    exe = str(tmp_path_factory.mktemp("streams") / "host_stream_order_check")
    # exported, the stand-ins come before the HIP runtime's own functions
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-std=c++17", "-O1", "-I",
                        os.path.join(ROOT, "include"),
                        os.path.join(ROOT, "tests", "host_stream_order_check.cpp"),
                        "-o", exe, "-rdynamic", "-pthread", "-ldl"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


@pytest.mark.parametrize("mode", ["same", "other", "release"])
def test_launches_of_calls_from_several_threads(checker, mode):
    r = subprocess.run([checker, _binding.LIB_PATH, mode], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr
    assert f"{mode}: 0 failure(s)" in r.stdout


def test_attention_kernel_of_queries_that_may_share_tokens(checker):
    r = subprocess.run([checker, _binding.LIB_PATH, "loads"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "loads: 0 failure(s)" in r.stdout, r.stdout + r.stderr
