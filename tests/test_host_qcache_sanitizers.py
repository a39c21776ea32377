"""Host AddressSanitizer + UndefinedBehaviorSanitizer run of the quantised cache's argument
checks and size query (CPU only; device code is built as usual, no sanitizer runs on the GPU).
host_qcache_abi_check.cpp says what is called."""
import concurrent.futures as cf
import os
import subprocess

import pytest

from test_host_sanitizers import HIPCC, HOST_SAN, ROOT, SAN_ENV

SOURCES = ["qcache_api", "qcache_attend"]


def test_quantised_cache_argument_checks_under_sanitizers(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not available")
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-fno-omit-frame-pointer", "-std=c++17",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I", os.path.join(ROOT, "include"), *HOST_SAN]
    sources = [os.path.join(ROOT, "prng_seeded_decode_amd", "csrc", s + ".hip") for s in SOURCES]
    sources.append(os.path.join(ROOT, "tests", "host_qcache_abi_check.cpp"))

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, *flags, "-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, f"{src}:\n{r.stderr[-3000:]}"
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(sources)) as ex:
        objs = list(ex.map(compile_one, sources))
    exe = str(tmp_path / "host_qcache_abi_check")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *HOST_SAN, *objs, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, env=dict(os.environ, **SAN_ENV),
                       timeout=100)
    log = r.stdout + r.stderr
    assert r.returncode == 0, log
    assert "quantised cache checks: 0 failure(s)" in log
    assert "ERROR: AddressSanitizer" not in log and "runtime error" not in log
