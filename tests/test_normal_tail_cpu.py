"""The normal distribution's tail as the feed-forward block's 16-bit kernels take it: the constants from
csrc/product_tile.h, evaluated in float32, against the true function; no GPU."""
import os
import re

import numpy as np
from scipy.special import erfc

from convolution_implicit_gemm_amd import build as B


def test_relative_error():
    source = open(os.path.join(B.CSRC, "product_tile.h")).read()
    body = re.search(r"float normal_fast\(float v, float& bell\) \{(.*?)\n\}", source, re.S)[1]
    f = np.float32
    number = r"(-?[\d.]+)f"
    exponent = f(re.search(rf"exp2f\({number} \* v \* v\)", body)[1])
    slope = f(re.search(rf"1\.0f \+ {number} \* fabsf\(v\)", body)[1])
    terms = [f(re.search(rf"float c = {number};", body)[1])] + [f(n) for n in re.findall(rf"c = c \* t \+ {number};", body)]
    assert len(terms) == 7
    v = np.linspace(0, 12.5, 250001).astype(f)
    t = f(1) / (f(1) + slope * v)
    c = np.full_like(v, terms[0])
    for term in terms[1:]:
        c = c * t + term
    bell = np.exp2((exponent * v * v).astype(np.float64)).astype(f)
    got = (c * (t * bell)).astype(np.float64)
    x = v.astype(np.float64)
    want = 0.5 * erfc(x / np.sqrt(2))
    assert np.all(np.abs(got / want - 1) < 4.2e-6 + 2.0 ** -23 * x * x)
    assert np.all(np.abs(bell / np.exp(-0.5 * x * x) - 1) < 2.0 ** -23 * (x * x + 1))
