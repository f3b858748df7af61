"""The fitted tail of the normal distribution behind GELU: the coefficients as the
header holds them, against erfc, and the accuracy that it states."""
import os
import re

import numpy as np
from scipy.special import erfcx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def source():
    with open(os.path.join(ROOT, "sparse_rank_linear_02_b200", "csrc", "epilogue.cuh")) as f:
        return f.read()


def coefficients():
    body = source().split("f32x2 normal_cdf2(")[1].split("float ta, tb;")[0]
    scale = float(re.search(r"fma2\(dup2\(([0-9.]+)f\), pack2\(fabsf", body).group(1))
    first = float(re.search(r"f32x2 q = dup2\((-?[0-9.e-]+)f\)", body).group(1))
    rest = [float(c) for c in re.findall(r"q = fma2\(q, t, dup2\((-?[0-9.e-]+)f\)\)", body)]
    return scale, [first] + rest


def test_the_tail_s_coefficients_are_as_close_as_stated():
    scale, c = coefficients()
    assert len(c) == 9 and all(float(np.float32(x)) == x for x in c)
    a = np.linspace(0.0, 13.5, 1_000_001)
    t = 1.0 / (1.0 + scale * a)
    tail = np.polyval(c, t) * t                       # of e^(-a^2 / 2)
    worst = np.abs(tail / (0.5 * erfcx(a / np.sqrt(2.0))) - 1.0).max()
    stated = float(re.search(r"relative error: ([0-9.e-]+) for a <= 13.5", source()).group(1))
    assert worst <= stated <= 1.1 * worst


def test_the_tail_in_fp32_is_as_close_as_stated():
    """The kernel's operations, each rounded to fp32; the approximate reciprocal and
    2^x add 2^-23 and 2^-22 (their bounds) to what is found here."""
    f = np.float32
    scale, c = coefficients()
    a = np.linspace(0.0, 13.0, 400_001).astype(f)
    d = a.astype(np.float64)
    fma = lambda x, y, z: (x.astype(np.float64) * y + z).astype(f)  # noqa: E731
    t = (1.0 / fma(a, np.float64(f(scale)), 1.0).astype(np.float64)).astype(f)
    q = np.full_like(a, f(c[0]))
    for x in c[1:]:
        q = fma(q, t, x)
    log2e = f(1.4426950408889634)
    arg = ((a * f(-0.5 * log2e)) * a).astype(np.float64)
    tail = ((q * t) * np.exp2(arg).astype(f)).astype(np.float64)
    err = np.abs(tail / (0.5 * erfcx(d / np.sqrt(2.0)) * np.exp(-d * d / 2)) - 1.0) + 2.0 ** -22 + 2.0 ** -23
    for top, stated in ((2.0, 1e-6), (4.0, 2e-6), (13.0, 1e-5)):
        assert err[d <= top].max() <= stated
