"""The polynomials of the score modifications as compiled (coefficients read from the source, rounded to
fp32) against their functions in fp64: the stated errors hold and are not far above the truth."""
import os
import re

import numpy as np
import pytest

from image_dits_b200 import build as rf2_build


def _source(name, start, end):
    text = open(os.path.join(rf2_build.CSRC, name)).read()
    return text[text.index(start):text.index(end, text.index(start))]


def _fp32_constants(code):
    """make_float2(c, c) pairs in the order of evaluation, highest power first."""
    pairs = re.findall(r"make_float2\((-?[0-9.]+)f, (-?[0-9.]+)f\)", code)
    assert all(a == b for a, b in pairs)
    return [float(np.float32(a)) for a, _ in pairs]


def _horner(c, u):
    p = np.full_like(u, c[0])
    for x in c[1:]:
        p = p * u + x
    return p


def test_tanh_up_to_the_cap():
    c = _fp32_constants(_source("score_mod.cuh", "float2 tanh_poly(", "\n}"))
    assert len(c) == 6
    x = np.linspace(1e-6, 1.0, 400001)
    err = np.abs(x * _horner(c, x * x) / np.tanh(x) - 1).max()
    assert 6.1e-7 <= err <= 6.2e-7


def test_tanh_up_to_half_the_cap():
    code = _source("rf2_lib.cu", "static const double c[4] = {", "}")
    c = [float(v) for v in re.findall(r"-?[0-9]+\.[0-9]+", code[code.index("{"):])]
    assert len(c) == 4
    x = np.linspace(1e-6, 0.5, 400001)
    for scale in (1.0, 0.0123):                  # as they are, and with a product's factors inside, rounded to fp32
        k = [float(np.float32(a * scale ** (2 * i + 1))) for i, a in enumerate(c)]
        y = x / scale
        err = np.abs(y * _horner(k[::-1], y * y) / np.tanh(x) - 1).max()
        assert err <= 6.2e-7, err                # 5.6e-7, and 2^-24 for the coefficients' rounding


def test_power_of_two():
    c = _fp32_constants(_source("ptx.cuh", "float2 ex2_poly(", "\n}"))
    c = [v for v in c if v != -1.0]              # -1: the reduced argument
    assert len(c) == 5
    r = np.linspace(-0.5, 0.5, 400001)
    err = np.abs(_horner(c, r) / np.exp2(r) - 1).max()
    assert 2.6e-6 <= err <= 2.7e-6


@pytest.mark.parametrize("x", [-126.0, -125.5, -60.25, -0.5, -0.49, 0.0, 0.5, 3.75, 99.0, float("nan")])
def test_power_of_two_as_computed(x):
    """The fp32 steps of ex2_poly: the exponent by adding 1.5 * 2^23, a NaN kept."""
    c = [np.float32(v) for v in _fp32_constants(_source("ptx.cuh", "float2 ex2_poly(", "\n}")) if v != -1.0]
    f = np.float32
    v = np.maximum(f(x), f(-126.0))              # numpy's maximum keeps NaN, as max.NaN does
    t = v + f(12582912.0)
    r = v - (t - f(12582912.0))
    p = c[0]
    for a in c[1:]:
        p = f(float(p) * float(r) + float(a))    # fused: one rounding (the product is exact in fp64)
    bits = (int(np.array(t, f).view(np.uint32)) << 23) + 0x3f800000 & 0xffffffff
    y = p * np.array(bits, np.uint32).view(f)
    assert np.isnan(y) if np.isnan(x) else abs(float(y) / 2.0 ** x - 1) <= 2.7e-6 + 2.0 ** -22
