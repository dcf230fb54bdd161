"""Host code of the 8-bit blocks under AddressSanitizer and
UndefinedBehaviorSanitizer: tests/sanitize/block_checks.cpp drives
csrc/block_args.cpp through refused and random sizes, block plans, and the rules
that choose a product's kernel, which it also pins for the GPU tests' shapes."""
import os
import shutil
import subprocess

import pytest

from test_host_sanitizers import ROCM_INCLUDE, ROOT, SAN, _run

CSRC = os.path.join(ROOT, "parameter_layout_collectives_amd", "csrc")
SOURCES = [os.path.join(CSRC, "plan.cpp"), os.path.join(CSRC, "block_args.cpp"),
           os.path.join(ROOT, "tests", "sanitize", "block_checks.cpp")]


def test_block_host_code_under_asan_and_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("needs g++ and the ROCm headers")
    exe = str(tmp_path / "block_checks")
    build = subprocess.run(
        [gxx, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE, *SAN, *SOURCES,
         "-o", exe], capture_output=True, text=True, timeout=600)
    assert build.returncode == 0, build.stderr[-4000:]
    _run(exe, "block checks passed")
