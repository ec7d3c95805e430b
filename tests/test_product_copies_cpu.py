"""The copies of the feed-forward block's tiles to LDS are assembly: the compiler does not know that
they read scalar registers, which a vector instruction must have written five wait states before.
Looks for that, and for scratch memory, in the listings of the units as they are built; no GPU."""
import concurrent.futures
import os
import re
import shutil
import subprocess

import pytest

from convolution_implicit_gemm_amd import build as B


def too_near(listing):
    """(copies, [(writer, copy)]) of a listing, function by function."""
    copies, found = 0, []
    for body in re.split(r"\n(?=_Z\w+:)", listing):
        lines = [line.strip() for line in body.splitlines()]
        lines = [line for line in lines if line and line[0] not in ";." and not line.endswith(":")]
        for i, line in enumerate(lines):
            m = re.match(r"buffer_load_dwordx4 v\d+, s\[(\d+):(\d+)\].* lds", line)
            if not m:
                continue
            copies += 1
            read, states = set(range(int(m[1]), int(m[2]) + 1)), 0
            for before in reversed(lines[max(0, i - 12):i]):
                if states >= 5:
                    break
                if before.startswith("s_nop"):
                    states += int(before.split()[1]) + 1
                    continue
                w = re.match(r"v_\S+\s+s(?:\[(\d+):(\d+)\]|(\d+)),", before)
                if w:
                    written = {int(w[3])} if w[3] else set(range(int(w[1]), int(w[2]) + 1))
                    if written & read:
                        found.append((before, line))
                states += 1
    return copies, found


def test_the_search_finds_one():
    text = "\n_Zk:\n\tv_readfirstlane_b32 s5, v1\n\ts_nop 2\n\tbuffer_load_dwordx4 v2, s[4:7], 0 offen lds\n"
    assert len(too_near(text)[1]) == 1
    assert too_near(text.replace("s_nop 2", "s_nop 4")) == (1, [])


def test_copies_wait_for_their_registers(tmp_path):
    if shutil.which("hipcc") is None:
        pytest.skip("hipcc not available")

    def listing(name):
        out = tmp_path / f"{name}.s"
        flags = [f for f in B.FLAGS if f != "-fPIC"]
        r = subprocess.run(["hipcc", *flags, "-S", "--cuda-device-only", "-x", "hip",
                            os.path.join(B.CSRC, f"kernels_gated_{name}.hip"), "-o", str(out)],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        return out.read_text()

    with concurrent.futures.ThreadPoolExecutor(3) as ex:
        for name, text in zip(("f32", "f16", "bf16"), ex.map(listing, ("f32", "f16", "bf16"))):
            copies, found = too_near(text)
            assert copies > 300 and not found, (name, copies, found[:3])
            scratch = [int(n) for n in re.findall(r"\.private_segment_fixed_size: (\d+)", text)]
            assert scratch and max(scratch) == 0, (name, scratch)
