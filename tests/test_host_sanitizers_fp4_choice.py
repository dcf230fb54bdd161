"""A 4-bit product runs with the workspace that it asks for as with any larger one:
tests/sanitize/fp4_choice_checks.cpp, under the sanitizers as test_host_sanitizers_fp4.py."""
import os
import shutil
import subprocess

import pytest

from test_host_sanitizers import ROCM_INCLUDE, ROOT, SAN, _run

CSRC = os.path.join(ROOT, "parameter_layout_collectives_amd", "csrc")
SOURCES = [os.path.join(CSRC, s) for s in ("plan.cpp", "block_args.cpp", "fp4_args.cpp")] + \
    [os.path.join(ROOT, "tests", "sanitize", "fp4_choice_checks.cpp")]


def test_the_asked_workspace_is_enough(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("needs g++ and the ROCm headers")
    exe = str(tmp_path / "fp4_choice_checks")
    build = subprocess.run(
        [gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE, *SAN, *SOURCES,
         "-o", exe], capture_output=True, text=True, timeout=600)
    assert build.returncode == 0, build.stderr[-4000:]
    _run(exe, "fp4 choice checks passed")
