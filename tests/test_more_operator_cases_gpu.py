"""perf/more_operators.py: its cases at reduced sizes and some drawn ones, by the library and by the
plain forms, against its 64-bit definition, and its counts of work."""
import math
import random
import sys

import pytest
import torch

from perf import more_operators as operators

pytestmark = pytest.mark.gpu


def small(c):
    """The case with sizes that its definition needs little time for."""
    c = dict(c)
    for name, most in (("b", 3), ("s", 300), ("m", 3000), ("c", 1032), ("f", 2744)):
        if name in c:
            c[name] = min(c[name], most)
    return c


def drawn():
    rng = random.Random(12)
    return [small(dict(operators.draw(rng), name=f"drawn{n}")) for n in range(40)]


CASES = [small(c) for c in operators.listed()] + drawn()


@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("c", CASES, ids=[c["name"] for c in CASES])
def test_case(c, own, monkeypatch):
    sys.__stderr__.write(f"CASE more operators own {own} {c}\n")
    sys.__stderr__.flush()
    monkeypatch.setattr(operators, "own", own)
    work = operators.work(c)
    assert work["bytes"] > 0 and work["flops"] >= 0
    got = operators.run(operators.prepare(c, 3))
    want = operators.exact(c, 3)
    torch.cuda.synchronize()
    got, want = ((v,) if torch.is_tensor(v) else v for v in (got, want))
    for a, b in zip(got, want, strict=True):
        assert a.shape == b.shape
        u = torch.finfo(a.dtype).eps / 2
        a = a.double()
        assert torch.isfinite(a).all()
        # results and up to two factors of a sum's products are rounded to T, each by u at most and
        # independently; float32 sums of up to 10^4 values of about 1 add 1e-5 of that
        error = (a - b).norm()
        assert error <= 3 * u * b.norm() + 1e-5 * (b.norm() + math.sqrt(b.numel())), float(error)
