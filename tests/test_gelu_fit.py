"""The gelu's polynomial as the source holds it, in 64 bits against erfcx and erfc (no GPU)."""
import math
import os
import re

import numpy as np
from scipy.special import erfcx

import genomic_lm_amd as G

SOURCE = os.path.join(os.path.dirname(G.__file__), "csrc", "linear_common.hpp")
BOUND = 3.5e-8               # relative, as the comment beside the coefficients says


def stored():
    """The argument's factor and the coefficients from the highest on, as the fp32 that they are."""
    text = open(SOURCE).read()
    text = text[text.index("ACT == ACT_GELU)"):text.index("ACT == ACT_GELU_TANH)")]
    number = r"(-?[0-9.]+)f"
    a, = re.findall(r"fmaf\(fabsf\(g\), " + number, text)
    q = re.findall(r"float q = " + number, text) + re.findall(r"q = fmaf\(q, t, " + number, text)
    return float(np.float32(a)), [float(np.float32(v)) for v in q]


def fitted(g):
    a, coefficients = stored()
    t, q = 1 / (1 + a * np.abs(g)), 0.0
    for c in coefficients:
        q = q * t + c
    return t * q


def test_the_coefficients_hold_the_stated_bound():
    assert len(stored()[1]) == 11
    g = np.concatenate([np.linspace(0, 30, 300001), np.logspace(1, 9, 100001)])
    assert np.abs(fitted(g) / erfcx(g / math.sqrt(2)) - 1).max() < BOUND
    assert "3.5e-8" in open(SOURCE).read()


def test_gelu_from_them():
    for g in np.linspace(-8, 8, 1601):
        h = 0.5 * math.exp(-g * g / 2) * fitted(g)
        got, want = (g * h if g < 0 else g * (1 - h)), 0.5 * g * math.erfc(-g / math.sqrt(2))
        assert abs(got - want) <= 1.1 * BOUND * abs(want) + 1e-300, g
