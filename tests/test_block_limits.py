"""The largest calls that complete a decoder block accepts and the first past them that it refuses
(block_abi.cpp), built for the host alone with the address and undefined-behaviour sanitizers
(tests/host_limits): an accepted call's launches stay below 2^32 threads and its offsets inside 32
bits.  No GPU."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_syrk_amd", "csrc")
ROCM_INC = "/opt/rocm/include"


def test_limits_under_host_sanitizers(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.isdir(ROCM_INC):
        pytest.skip("needs g++ and the ROCm headers")
    exe = str(tmp_path / "drive_limits")
    flags = ["-std=c++17", "-g", "-O1", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
             "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM_INC}", f"-I{CSRC}",
             f"-I{os.path.join(ROOT, 'include')}"]
    srcs = [os.path.join(CSRC, "block_abi.cpp"), os.path.join(ROOT, "tests", "host_limits", "drive_limits.cpp")]
    r = subprocess.run([cxx, *flags, *srcs, "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    out = r.stdout + r.stderr
    print(out[-2000:])
    assert r.returncode == 0 and " 0 failed" in r.stdout, out[-4000:]
