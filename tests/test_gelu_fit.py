"""CPU: the constants of the kernels' gelu (csrc/epilogue.hpp), read from the source, against the function that
they fit: Q(t) = erfcx(x) / (2 t), t = 1 / (1 + 0.42 x), x = |v| / sqrt 2, 0 <= x <= 9.5, is met with the
largest relative error that the source states, and no polynomial of its degree does much better."""
import math
import os
import re

import numpy as np
import pytest

special = pytest.importorskip("scipy.special")

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fine_grained_block_amd", "csrc",
                   "epilogue.hpp")


def _constants():
    text = open(SRC).read()
    body = re.search(r"float gelu_erf\(float v\) \{(.*?)\n\}", text, re.S).group(1)
    scale = float(re.search(r"fmaf\(([\d.]+)f, fabsf\(v\), 1\.0f\)", body).group(1))
    top = float(re.search(r"float q = ([-\d.]+)f;", body).group(1))
    rest = [float(c) for c in re.findall(r"q = __builtin_fmaf\(q, t, ([-\d.]+)f\);", body)]
    rate = float(re.search(r"exp2f\(v \* v \* ([-\d.]+)f\)", body).group(1))
    stated = float(re.search(r"largest relative error ([\d.]+e-\d+) with the constants as they are", text).group(1))
    return scale, [top] + rest, rate, stated


def test_fit_against_erfcx():
    scale, coef, rate, stated = _constants()
    assert len(coef) == 8 and scale == pytest.approx(0.42 / math.sqrt(2), rel=1e-7)
    assert rate == pytest.approx(-0.5 / math.log(2), rel=1e-7)
    x = np.linspace(0.0, 9.5, 200001)
    t = 1.0 / (1.0 + 0.42 * x)
    want = special.erfcx(x) / (2 * t)
    err = np.abs(np.polyval(coef, t) / want - 1)
    assert 0.9 * stated < err.max() <= stated
    # the best of degree 7 at these points, by reweighted least squares (each step raises the weights where the
    # error is large): no polynomial's largest error is below the weighted mean error of such a step
    t, want = t[::50], want[::50]
    w = np.full(t.size, 1.0 / t.size)
    low = 0.0
    for _ in range(60):
        a = np.polynomial.chebyshev.chebvander((2 * t - t.min() - 1) / (1 - t.min()), 7) / want[:, None]
        c = np.linalg.lstsq(a * np.sqrt(w)[:, None], np.sqrt(w), rcond=None)[0]
        e = np.abs(a @ c - 1)
        low = max(low, math.sqrt(np.sum(w * e * e)))
        w = w * e
        w /= w.sum()
    assert low > 0.5 * err.max(), (low, err.max())


def test_gelu_of_the_fit():
    """The kernel's formula in 64 bits: within 1e-6 relative of v Phi(v) for |v| < 4, exact limits."""
    scale, coef, rate, _ = _constants()
    v = np.linspace(-4, 4, 100001)
    t = 1.0 / (1.0 + scale * np.abs(v))
    h = np.minimum(v, 16.0) * np.polyval(coef, t) * t * np.exp2(v * v * rate)
    got = np.where(v < 0, h, v - h)
    want = 0.5 * v * special.erfc(-v / math.sqrt(2))
    assert np.all(np.abs(got - want) <= 1e-6 * np.abs(want))
