"""The polynomials of the feed-forward block's gelu (normal_tail in csrc/ffn.cu): the normal distribution's
function at -u over exp(-u^2 / 2), in t = 1 / (1 + 0.3 u)."""
import math
import os
import re

import numpy as np
import pytest

from conftest import ROOT

U = np.linspace(0, 14.5, 8001)
T = 1 / (1 + 0.3 * U)
TAIL = np.array([0.5 * math.erfc(u / math.sqrt(2)) * math.exp(u * u / 2) for u in U])


def _polynomials():
    text = open(os.path.join(ROOT, "exact_dimensional_distance_gb300", "csrc", "ffn.cu")).read()
    body = text[text.index("float2 normal_tail("):]
    body = body[:body.index("return r;")]
    number = r"(-?\d\.\d+e[-+]\d+)f"
    fast, full = body[body.index("if (FAST)"):].split("} else {")
    return {name: [float(v) for v in re.findall(number, part)] for name, part in (("fast", fast), ("full", full))}


def _fit(degree):
    """The smallest largest relative error that least squares reach whose weights grow with the error (Lawson)."""
    rows = np.vander(T, degree + 1) / TAIL[:, None]
    weight, best = np.ones_like(T), np.inf
    for _ in range(300):
        s = np.sqrt(weight)
        error = np.abs(rows @ np.linalg.lstsq(rows * s[:, None], s, rcond=None)[0] - 1)
        best = min(best, error.max())
        weight *= error
        weight /= weight.sum()
    return best


@pytest.mark.parametrize("name,degree,stated", [("fast", 6, 2.2e-6), ("full", 8, 4e-7)])
def test_polynomial_is_the_best_fit(name, degree, stated):
    c = _polynomials()[name]
    assert len(c) == degree + 1
    error = np.abs(np.polyval(c, T) / TAIL - 1).max()
    assert error <= 1.25 * _fit(degree)
    # in float32: at each step half a unit of the sum, and of t, on top
    t, r = T.astype(np.float32), np.full(T.shape, c[0], dtype=np.float32)
    for v in c[1:]:
        r = (r.astype(np.float64) * t + np.float32(v)).astype(np.float32)  # one rounding
    assert np.abs(r / TAIL - 1).max() <= stated
