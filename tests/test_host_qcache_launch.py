"""What seedlm_qcache_attend launches for a call's sizes, on the CPU; host_qcache_launch_check.cpp
says what is checked."""
import concurrent.futures as cf
import os
import subprocess

import pytest

from test_host_sanitizers import HIPCC, ROOT

FLAGS = ["--offload-arch=gfx950", "-O1", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
         "-packed-fp32-ops", "-I", os.path.join(ROOT, "include")]


def test_rows_of_one_token_a_request_launch_what_no_rows_do(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not available")
    csrc = os.path.join(ROOT, "prng_seeded_decode_amd", "csrc")
    sources = [os.path.join(csrc, "qcache_api.hip"), os.path.join(csrc, "qcache_attend.hip"),
               os.path.join(ROOT, "tests", "host_qcache_launch_check.cpp")]

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, *FLAGS, "-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, f"{src}:\n{r.stderr[-3000:]}"
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(sources)) as ex:
        objs = list(ex.map(compile_one, sources))
    exe = str(tmp_path / "host_qcache_launch_check")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *objs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "0 failure(s)" in r.stdout
