"""The host code of layer norm, rotary and attention under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU): transformer_sanitizer_driver.cpp sweeps descriptions, with values
from the ends of their ranges among them, through create, workspace size and destroy, and checks that
each attention kernel's LDS limit is set to one size.  Both sanitizers apply to the host pass only; the device pass, at -O0, just gives the objects their code.
"""
import concurrent.futures
import os
import shutil
import subprocess

import pytest

from convolution_implicit_gemm_amd import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANGXX = "/opt/rocm/llvm/bin/clang++"
SAN = ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=undefined"]
HOST_FLAGS = ["-O1", "-g", "-std=c++17", "-fPIC", "-fno-omit-frame-pointer", "-I", B.INCLUDE, "-I", B.CSRC]
SOURCES = ["transformer.cpp", "kernels_layernorm.hip", "kernels_rotary.hip", "kernels_attention_d128.hip",
           "kernels_attention_d96.hip", "kernels_attention_d64.hip", "kernels_attention_d32.hip"]


def test_host_code_under_asan_and_ubsan(tmp_path):
    if shutil.which("hipcc") is None or not os.path.exists(CLANGXX):
        pytest.skip("hipcc / ROCm clang not available")

    def compile_one(src):
        obj = str(tmp_path / (os.path.splitext(src)[0] + ".o"))
        if src.endswith(".hip"):
            host_only = [x for f in SAN for x in ("-Xarch_host", f)]
            cmd = ["hipcc", f"--offload-arch={B.ARCH}", *HOST_FLAGS, "-Xarch_device", "-O0", "-Xarch_device", "-g0",
                   *host_only, "-x", "hip", "-c", os.path.join(B.CSRC, src), "-o", obj]
        else:
            cmd = [CLANGXX, *HOST_FLAGS, *SAN, "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-c",
                   os.path.join(B.CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    exe = str(tmp_path / "driver")
    r = subprocess.run([CLANGXX, *HOST_FLAGS, *SAN, "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                        os.path.join(ROOT, "tests", "transformer_sanitizer_driver.cpp"), *objs, "-L/opt/rocm/lib",
                        "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe, "60000"], capture_output=True, text=True, env=env, timeout=600)
    report = r.stdout + r.stderr
    assert r.returncode == 0, report[-4000:]
    assert "runtime error" not in report and "AddressSanitizer" not in report, report[-4000:]
    created, rejected, kernels = (int(r.stdout.split()[n]) for n in (1, 3, 5))
    assert created > 80000 and rejected > 30000, r.stdout
    assert kernels == 24, r.stdout  # two forms, three types, four head sizes
