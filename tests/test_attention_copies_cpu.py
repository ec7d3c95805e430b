"""The compiler has to know that a copy to LDS goes by m0: between two copies of its own to one
address it keeps the register, unless it sees the other one's value.  Compiles a kernel; no GPU."""
import re
import shutil
import subprocess

import pytest

from convolution_implicit_gemm_amd import build as B

KERNEL = r"""
#include "attention_tile.h"
extern "C" __global__ void probe(const float* p, float* out, int at) {
  extern __shared__ __attribute__((aligned(16))) float lds[];
  typedef const __attribute__((address_space(1))) void* from_t;
  typedef __attribute__((address_space(3))) void* to_t;
  to_t to = (to_t)(lds + at);
  __builtin_amdgcn_global_load_lds((from_t)(p + threadIdx.x), to, 4, 0, 0);
  fc::copy_to_lds<4>(fc::lds_offset(lds + 512), threadIdx.x * 4, p + 64);
  __builtin_amdgcn_global_load_lds((from_t)(p + 128 + threadIdx.x), to, 4, 0, 0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  out[threadIdx.x] = lds[threadIdx.x] + lds[512 + threadIdx.x];
}
"""


@pytest.mark.parametrize("level", ["-O3", "-O0"])
def test_every_copy_has_its_own_address(tmp_path, level):
    if shutil.which("hipcc") is None:
        pytest.skip("hipcc not available")
    source, listing = tmp_path / "probe.hip", tmp_path / "probe.s"
    source.write_text(KERNEL)
    flags = [f for f in B.FLAGS if f not in ("-O3", "-fPIC")]
    r = subprocess.run(["hipcc", *flags, level, "-S", "--cuda-device-only", "-x", "hip", str(source), "-o",
                        str(listing)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    body = listing.read_text().split("\nprobe:")[1].split("s_endpgm")[0]
    set_since = False
    copies = 0
    for line in body.splitlines():
        if re.search(r"\bm0\b", line) and re.match(r"\s*s_\w+ m0\b", line):
            set_since = True
        elif "global_load_lds_dword" in line:
            assert set_since, f"copy {copies} goes where the last one went:\n{body}"
            set_since, copies = False, copies + 1
    assert copies == 3, body
