"""The polynomial of the normal distribution's tail in gelu, read from the kernels' header, against erfc in 64 bits: the polynomial
itself, and the header's steps in fp32 against the bound that it states.  No GPU.

Tolerances: 5.1e-8 is what the header states of the stored coefficients (5.0e-8, and the grid's own step); a coefficient off by
1e-5 of itself moves q by 2e-7 of itself or more somewhere.  In fp32 steps the header states (a^2 + 10) 2^-24, with a unit in the last
place of either sign each from the hardware's reciprocal and exponential."""
import os
import re

import numpy as np
import pytest
from scipy.special import erfcx

import segmented_gather_matvec_amd as sg

f32 = np.float32


def numbers():
    src = open(os.path.join(os.path.dirname(sg.__file__), "csrc", "sgmv_layer_ops.h")).read()
    body = src[src.index("float normal_tail("):]
    body = body[: body.index("\n}")]
    scale = re.search(r"fmaf\(a, (0\.\d+)f, 1\.f\)", body).group(1)
    exponent = re.search(r"exp2f\((-0\.\d+)f \* \(a \* a\)\)", body).group(1)
    q = re.findall(r"float q = (-?0\.\d+)f;", body) + re.findall(r"fmaf\(q, t, (-?0\.\d+)f\)", body)
    assert len(q) == 9 and body.count("fmaf(q, t,") == 8
    return f32(scale), f32(exponent), [f32(v) for v in q]


def polynomial_error(scale, q):
    a = np.linspace(0, 15, 1000001)
    t = 1 / (1 + float(scale) * a)
    value = np.full_like(a, float(q[0]))
    for k in q[1:]:
        value = value * t + float(k)
    return np.abs(t * value / (0.5 * erfcx(a / np.sqrt(2))) - 1).max()


def test_polynomial():
    scale, exponent, q = numbers()
    assert abs(float(exponent) + 0.5 / np.log(2)) <= 2.0 ** -25
    assert polynomial_error(scale, q) < 5.1e-8


@pytest.mark.parametrize("which", range(9))
def test_a_coefficient_beside_its_value_shows(which):
    """(The oracle's own copy of the numbers is changed, not the header.)"""
    scale, _, q = numbers()
    q = [float(v) * (1 + 1e-5) if i == which else float(v) for i, v in enumerate(q)]
    assert polynomial_error(scale, q) > 1e-7


@pytest.mark.parametrize("recip,power", [(0, 0), (1, 1), (-1, -1), (1, -1), (-1, 1)])
def test_steps_in_fp32(recip, power):
    scale, exponent, q = numbers()
    rng = np.random.default_rng(3)
    a = np.concatenate([np.linspace(0, 13, 300001), rng.uniform(0, 13, 300000)]).astype(f32)

    def fma(x, y, z):       # (a product of two fp32 numbers is exact in 64 bits)
        return (x.astype(np.float64) * y + np.float64(z)).astype(f32)

    def moved(x, units):
        return np.nextafter(x, f32(np.inf if units > 0 else -np.inf)) if units else x

    t = moved((1 / fma(a, np.float64(scale), 1.0).astype(np.float64)).astype(f32), recip)
    E = moved(np.exp2((exponent * (a * a)).astype(np.float64)).astype(f32), power)
    value = np.full_like(a, q[0])
    for k in q[1:]:
        value = fma(value, t.astype(np.float64), k)
    got = (E * t * value).astype(np.float64)
    x = a.astype(np.float64)
    want = 0.5 * erfcx(x / np.sqrt(2)) * np.exp(-x * x / 2)
    assert (np.abs(got / want - 1) <= (x * x + 10) * 2.0 ** -24).all()
