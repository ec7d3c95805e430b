"""The host code behind include/fusedconv_block.h under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU): block_sanitizer_driver.cpp sweeps descriptions, with values from the
ends of their ranges among them, through create, workspace size, the checks of a call and destroy."""
import os
import subprocess

import pytest

from convolution_implicit_gemm_amd import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANGXX = "/opt/rocm/llvm/bin/clang++"
SAN = ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=undefined"]


def test_host_code_under_asan_and_ubsan(tmp_path):
    if not os.path.exists(CLANGXX):
        pytest.skip("ROCm clang not available")
    exe = str(tmp_path / "driver")
    r = subprocess.run([CLANGXX, "-O1", "-g", "-std=c++17", "-fno-omit-frame-pointer", *SAN, "-D__HIP_PLATFORM_AMD__",
                        "-I", "/opt/rocm/include", "-I", B.INCLUDE, "-I", B.CSRC,
                        os.path.join(ROOT, "tests", "block_sanitizer_driver.cpp"), os.path.join(B.CSRC, "block.cpp"),
                        os.path.join(B.CSRC, "gated_plan.cpp"), "-L/opt/rocm/lib", "-lamdhip64",
                        "-Wl,-rpath,/opt/rocm/lib", "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe, "60000"], capture_output=True, text=True, env=env, timeout=600)
    report = r.stdout + r.stderr
    assert r.returncode == 0, report[-4000:]
    assert "runtime error" not in report and "AddressSanitizer" not in report, report[-4000:]
    created, rejected, launched = (int(r.stdout.split()[n]) for n in (1, 3, 5))
    assert created > 80000 and rejected > 15000 and launched > 80000, r.stdout
