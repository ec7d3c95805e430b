"""perf/operators.py: its cases at reduced sizes and some drawn ones, by the library and by the plain
forms, against its 64-bit definition, and its counts of work."""
import math
import random
import sys

import pytest
import torch

from perf import operators

pytestmark = pytest.mark.gpu


def small(c):
    """The case with a batch, lengths and planes that its definition needs little time for."""
    c = dict(c)
    for name, most in (("n", 3), ("b", 3), ("sq", 700), ("sk", 1500), ("s", 100), ("inner", 4096)):
        if name in c:
            c[name] = min(c[name], most)
    if c.get("packed") and "sq" in c:
        c["sk"] = c["sq"]
    return c


def drawn():
    rng = random.Random(11)
    return [small(dict(operators.draw(rng), name=f"drawn{n}")) for n in range(40)]


CASES = [small(c) for c in operators.listed()] + drawn()


@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("c", CASES, ids=[c["name"] for c in CASES])
def test_case(c, own, monkeypatch):
    sys.__stderr__.write(f"CASE operators own {own} {c}\n")
    sys.__stderr__.flush()
    monkeypatch.setattr(operators, "own", own)
    work = operators.work(c)
    assert work["bytes"] > 0 and work["flops"] >= 0
    got = operators.run(operators.prepare(c, 3))
    want = operators.exact(c, 3)
    torch.cuda.synchronize()
    u = torch.finfo(operators.TYPES[c["dtype"]]).eps / 2
    for a, b in zip(got, want, strict=True):
        assert a.shape == b.shape
        a = a.double()
        fine = torch.isfinite(b)
        assert torch.equal(fine, torch.isfinite(a))
        # results and up to two factors of a sum's products are rounded to T, each by u at most and
        # independently; float32 sums of up to 10^4 values of about 1 add 1e-5 of that
        error = (a - b)[fine].norm()
        assert error <= 3 * u * b[fine].norm() + 1e-5 * (b[fine].norm() + math.sqrt(b.numel())), float(error)
