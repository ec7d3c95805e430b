"""An unoptimised build of the feed-forward block's kernels makes the copies to LDS that the library's
does, and each waits for its scalar registers; no GPU."""
import os
import shutil
import subprocess

import pytest

from convolution_implicit_gemm_amd import build as B
from tests.test_product_copies_cpu import too_near


def test_the_same_copies(tmp_path):
    if shutil.which("hipcc") is None:
        pytest.skip("hipcc not available")
    out = tmp_path / "unit.s"
    flags = [f for f in B.FLAGS if f not in ("-fPIC", "-O3")]
    r = subprocess.run(["hipcc", *flags, "-O0", "-S", "--cuda-device-only", "-x", "hip",
                        os.path.join(B.CSRC, "kernels_gated_f32.hip"), "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    copies, found = too_near(out.read_text())
    assert copies > 100 and not found, (copies, found[:3])
