"""The host half of the state space block's library (argument checks, extents, overlaps, the plans of
chunks and tiles) under AddressSanitizer and UndefinedBehaviorSanitizer: rebuilt with both, and
test_ssm_abi.py run against it in a child process. Device code is compiled without optimization and
never launched."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from masked_depthwise_causal_amd import build

from .test_sanitizers import ROOT, _asan_runtime


@pytest.mark.slow
def test_host_side_clean_under_asan_and_ubsan(tmp_path):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    rt = _asan_runtime()
    if not (os.path.exists(hipcc) and rt):
        pytest.skip("hipcc or the clang sanitizer runtime not available")
    flags = [hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
             "-Xarch_device", "-O0", "-Xarch_device", "-g0",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
             "-I", build.INCLUDE]
    jobs = [(str(tmp_path / (os.path.basename(s) + ".o")), s) for s in build.SSM_SRCS]
    running = [subprocess.Popen([*flags, "-c", s, "-o", o], stderr=subprocess.PIPE, text=True)
               for o, s in jobs]
    for p in running:
        err = p.communicate(timeout=1200)[1]
        assert p.returncode == 0, err[-4000:]
    lib = str(tmp_path / "libmccb_ssm_san.so")
    res = subprocess.run([*flags, "-shared", *(o for o, _ in jobs), "-o", lib], capture_output=True,
                         text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    env = dict(os.environ, LD_PRELOAD=rt, MCCB_SSM_LIBRARY=lib,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    run = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "not gpu", "-p",
                          "no:cacheprovider", "tests/test_ssm_abi.py", "-k",
                          "not struct_sizes and not front_end"], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=1200)
    out = run.stdout + run.stderr
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-6000:]
    assert run.returncode == 0, out[-6000:]
    assert " passed" in run.stdout
