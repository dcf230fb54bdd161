"""Host code of the 4-bit blocks and of the orthogonalised updates under
AddressSanitizer and UndefinedBehaviorSanitizer: tests/sanitize/fp4_checks.cpp drives
csrc/fp4_args.cpp and csrc/ortho_args.cpp through refused and random sizes."""
import os
import shutil
import subprocess

import pytest

from test_host_sanitizers import ROCM_INCLUDE, ROOT, SAN, _run

CSRC = os.path.join(ROOT, "parameter_layout_collectives_amd", "csrc")
SOURCES = [os.path.join(CSRC, s) for s in ("plan.cpp", "block_args.cpp", "fp4_args.cpp",
                                           "ortho_args.cpp")] + \
    [os.path.join(ROOT, "tests", "sanitize", "fp4_checks.cpp")]


def test_fp4_and_ortho_host_code_under_asan_and_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("needs g++ and the ROCm headers")
    exe = str(tmp_path / "fp4_checks")
    build = subprocess.run(
        [gxx, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE, *SAN, *SOURCES,
         "-o", exe], capture_output=True, text=True, timeout=600)
    assert build.returncode == 0, build.stderr[-4000:]
    _run(exe, "fp4 checks passed")
