"""The fit behind gelu (CPU only): the coefficients in csrc/linear.hip hold the
bounds that the comment beside them states."""

import os
import re

import numpy as np
from scipy import special

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def constants():
    src = open(os.path.join(ROOT, "rank_step_amd", "csrc", "linear.hip")).read()
    body = src[src.index("void normal(float z"):]
    body = body[:body.index("tail = p")]
    k = float(np.float32(re.search(r"fmaf\(([0-9.]+)f, fabsf", body).group(1)))
    c = [float(np.float32(v)) for v in re.findall(r"(?:p = |t, )(-?[0-9.]+)f", body)]
    assert len(c) == 9
    return k, c


def f32(v):
    return np.asarray(v).astype(np.float32).astype(np.float64)


def half_erfcx(z, off=None):
    """t P(t) in float64, or (off: the reciprocal's error in units of its last
    place) with every step rounded to fp32."""
    k, c = constants()
    r = f32 if off is not None else np.asarray
    t = r(1 / r(1 + k * z))
    if off:
        t = t + off * np.spacing(t.astype(np.float32)).astype(np.float64)
    p = np.full_like(t, c[0])
    for v in c[1:]:
        p = r(p * t + v)
    return r(p * t)


def points(hi):
    return f32(np.concatenate([np.linspace(0, min(hi, 1e3), 300001), np.geomspace(1e-6, hi, 100001)]))


def test_fit():
    z = points(1e30)
    assert np.abs(half_erfcx(z) / (special.erfcx(z / np.sqrt(2)) / 2) - 1).max() < 2.1e-7


def test_fit_in_fp32():
    z = points(13.3)
    ref = special.erfcx(z / np.sqrt(2)) / 2
    assert np.abs(half_erfcx(z, 0) / ref - 1).max() < 4.6e-7
    # A reciprocal within one unit of its last place is off by half a unit more,
    # 2^-24 of t at most; d ln g / d ln t is largest at t = 1, where g = 1 and
    # dg/dt = (2 / sqrt(pi)) / 0.4 = 2.83.
    for off in (-0.5, 0.5):
        assert np.abs(half_erfcx(z, off) / ref - 1).max() < 4.6e-7 + 2.83 * 2.0 ** -24, off


def test_lower_tail():
    """The tail's relative error grows like z^2, by the rounding of the exponent."""
    z = points(13.0)
    e = np.exp2(f32(f32(z * z) * f32(-0.5 * f32(1.44269504))))
    rel = np.abs(half_erfcx(z, 0) * e / special.ndtr(-z) - 1)
    assert np.all(rel < 4.6e-7 + z * z * 2.0 ** -24)
    assert rel[z < 5].max() > 1.2e-6 and rel[z < 8].max() > 2.5e-6
