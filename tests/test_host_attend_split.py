"""The attention kernels' split of units into runs (attend_split.h), on the CPU;
host_attend_split_check.cpp says what is checked."""
import os
import subprocess

import pytest

from test_host_sanitizers import HIPCC, ROOT


def test_runs_follow_one_another_and_none_is_empty(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not available")
    exe = str(tmp_path / "host_attend_split_check")
    r = subprocess.run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O2", "-std=c++17", "-Xclang",
                        "-target-feature", "-Xclang", "-packed-fp32-ops", "-I",
                        os.path.join(ROOT, "include"),
                        os.path.join(ROOT, "tests", "host_attend_split_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "0 failure(s)" in r.stdout
