"""Calls of several host threads on one stream (CPU only): host_stream_order_check.cpp loads the
built library on top of a stand-in for the HIP runtime and looks at the order of its launches."""
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
