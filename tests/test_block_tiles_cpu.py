"""tests/test_gated_ffn_tiles_gpu.py without a GPU: its sizes take every kernel of the feed-forward block's
products in each type, whole and split, and its distances resolve a missing stage of terms."""
import pytest
import torch

from tests.test_block_plans_cpu import FORMS, plans  # noqa: F401 (a fixture)
from tests.test_gated_ffn_tiles_gpu import SHAPES, TYPES, apart, distance_limit


def test_every_kernel_of_every_type(plans):  # noqa: F811
    got = plans([(list(TYPES).index(s[0]), *s[1:]) for s in SHAPES])
    for dtype in TYPES:
        seen = set()
        for (head, forms), shape in zip(got, SHAPES):
            if shape[0] != dtype:
                continue
            for name, (rows, cols, whole, splits, _, _) in forms.items():
                if head[0] and name in ("gate", "down"):
                    continue
                seen.update({(name, rows, cols, "whole")} if whole else ())
                seen.update({(name, rows, cols, "split")} if splits > 1 else ())
        tiles = [(256, 128), (128, 128), (64, 128)]
        want = {(n, *t, kind) for n in FORMS for t in tiles for kind in ("whole", "split")}
        if dtype != "f32":
            want |= {(n, 256, 256, kind) for n in FORMS if n != "hidden" for kind in ("whole", "split")}
        assert seen == want, (dtype, want ^ seen)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_distances_resolve_a_stage(dtype):
    """A weight's gradient without the last stage of rows, and one of zeros, at every number of rows (with
    few columns: the distance does not depend on them)."""
    t = TYPES[dtype]
    stage = 64 // torch.finfo(t).bits * 8 if dtype != "f32" else 16
    for _, m, c, f, o in (s for s in SHAPES if s[0] == dtype):
        g = torch.Generator().manual_seed(m)
        d, x = (torch.randn(m, 12, generator=g).to(t).double() for _ in range(2))
        want = d.T @ x
        most = distance_limit(t, max(m, c, 2 * f, o))
        assert apart(want.to(t), want) < most
        assert apart(torch.zeros_like(want), want) > most
        assert apart(d[:-stage].T @ x[:-stage], want) > most, (m, most)
