"""The stated error of the normal distribution's tail, of the polynomial in the source evaluated step by
step in fp32 with an exact power and reciprocal."""
import math
import os
import re

import numpy as np
from scipy.special import erfc

from orthogonalizing_polynomial_cascade_amd import build

F32 = np.float32


def _source():
    text = open(os.path.join(build.CSRC, "activation.h")).read()
    body = text[text.index("normal_cdf(float z"):]
    fit = [F32(v) for v in re.findall(r"(?:float r = |fmaf\(r, t, )(-?[\d.]+)f", body)]
    slope = F32(re.search(r"fmaf\(([\d.]+)f, fabsf\(z\)", body).group(1))
    power = F32(re.search(r"exp2f\(-([\d.]+)f \* z \* z\)", text).group(1))
    return fit, slope, power


def _fma(a, b, c):
    return (a.astype(np.float64) * np.float64(b) + np.float64(c)).astype(F32)


def _tail(z):
    fit, slope, power = _source()
    assert len(fit) == 9
    g = np.exp2(((-power * z).astype(F32) * z).astype(np.float64)).astype(F32)
    t = (1.0 / _fma(np.abs(z), slope, 1.0)).astype(F32)
    r = np.full_like(z, fit[0])
    for c in fit[1:]:
        r = _fma(r, t, c)
    return (F32(0.5) * t * r * g).astype(np.float64)


def test_tail_error():
    z = np.linspace(-13, 13, 1000001).astype(F32)
    want = 0.5 * erfc(np.abs(z).astype(np.float64) / math.sqrt(2.0))
    error = np.abs(_tail(z) - want) / want
    assert (error <= 5e-7 + 6e-8 * z.astype(np.float64) ** 2).all()
    assert error[np.abs(z) > 9].max() > 4e-6   # it does grow with z^2
