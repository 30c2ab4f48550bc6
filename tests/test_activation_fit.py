"""CPU: the polynomial behind the epilogue's gelu, with the coefficients as the kernel source
holds them, against the normal distribution function, and its fp32 evaluation with exp2 and
reciprocal rounded to nearest (the hardware's are within 1 ulp). The bounds are the figures
that the source states."""
import os
import re

import numpy as np
from scipy.special import erfcx, ndtr

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "fp8_block_scaled_dg_amd", "csrc",
                      "activation.hpp")
F = np.float32


def coefficients():
    """(c of t = 1 / (1 + c z), the polynomial's coefficients, highest power first)."""
    text = open(SOURCE).read()
    body = text[text.index("float act_tail("):]
    num = [F(x) for x in re.findall(r"(-?\d+\.\d+)f", body[:body.index("\n}\n")])]
    return num[0], num[1:]


def fma(a, b, c):
    """a * b + c of fp32 values, rounded once (to fp64 first: twice in rare cases)."""
    return (np.float64(a) * np.float64(b) + np.float64(c)).astype(F)


def test_fit():
    c, p = coefficients()
    y = np.linspace(0, 12, 200001)
    t = 1 / (1 + float(c) * y * np.sqrt(2))
    assert len(p) == 9 and np.max(np.abs(2 * t * np.polyval([float(x) for x in p], t) / erfcx(y) - 1)) < 4.9e-8


def test_fp32_tail():
    c, p = coefficients()
    z = np.linspace(0, 13, 400001).astype(F)
    t = (F(1) / fma(c, z, F(1))).astype(F)
    q = np.full_like(z, p[0])
    for x in p[1:]:
        q = fma(q, t, x)
    q = fma(q, t, F(0))
    q *= np.exp2((F(-0.5) * F(1.4426950408889634) * z * z).astype(np.float64)).astype(F)
    far = np.abs(q.astype(np.float64) / ndtr(-z.astype(np.float64)) - 1)
    assert np.max(far[z < 3]) < 7e-7 and np.max(far) < 8.2e-6
