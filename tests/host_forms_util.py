"""The plans of the 4-bit product with its epilogue (csrc/linear_plan.h, csrc/w4_plan.h), built for
the host with g++ and asked (tests/host_forms)."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_syrk_amd", "csrc")
DRIVER = os.path.join(ROOT, "tests", "host_forms", "drive_forms.cpp")


def build(folder) -> str:
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs g++")
    exe = str(folder / "drive_forms")
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", f"-I{CSRC}", DRIVER, "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    return exe


def ask(exe, cases):
    """cases of (m, d_out, d_in, group, gated); the line that the driver prints for each."""
    r = subprocess.run([exe, *(str(int(v)) for c in cases for v in c)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = r.stdout.splitlines()
    assert len(lines) == len(cases)
    return lines
