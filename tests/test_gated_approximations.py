"""The gated experts' activations as the kernels compute them (csrc/gated.cuh: approximate exponential and reciprocal
instructions, gelu's distribution function by a polynomial), step by step in fp32 without a GPU, against 64 bits.  The
instructions themselves are off by 2^-22 (ex2) and 2^-23 (rcp) of their results at most, which each bound adds.

Bounds, u = 2^-24.  A power's argument y is made by one rounding for silu, two for Phi and four for the tanh form (x^2, the
fused sum, the product; the constants' own), each of u of it, and a constant rounded to u / 2: an error of d in y is one
of d ln 2 of 2^y.  |y| ln 2 is |x|, x^2 / 2 and 1.6 |x| + 0.072 |x|^3.  What is left of the sums and products is a few u."""
import os
import re

import numpy as np
import pytest
import torch

from tests.gated_util import ACTS, act_error
from tests.test_warp_convergence import CSRC

F = np.float32
U = 2.0 ** -24


def _constants():
    with open(os.path.join(CSRC, "gated.cuh")) as f:
        text = f.read()
    named = {n: F(v) for n, v in re.findall(r"(k\w+) = ([\d.]+)f", text)}
    phi = text[text.index("float phi_of("):text.index("const float below")]
    scale = F(re.search(r"fmaf\(([\d.]+)f, fabsf\(x\)", phi).group(1))
    poly = [F(re.search(r"float r = ([\d.-]+)f", phi).group(1))] + [F(c) for c in re.findall(r"r = fmaf\(r, t, (-?[\d.]+)f\)", phi)]
    assert len(poly) == 8
    return named, scale, poly


def _fma(a, b, c):
    return F(a.astype(np.float64) * np.float64(b) + np.float64(c))  # the product of two fp32 is exact in 64 bits


def _exp2(y):
    return F(np.exp2(y.astype(np.float64)))


def _rcp(x):
    return F(1.0 / x.astype(np.float64))


def _factor(x, name):
    """act(x) / x as the kernels have it."""
    k, scale, poly = _constants()
    if name == "silu":
        return _rcp(F(1) + _exp2(F(-k["kLog2e"] * x)))
    if name == "gelu_tanh":
        y = F(x * _fma(F(x * x), F(-k["kTanh3"] * k["kLog2e"]), F(-k["kTanh"] * k["kLog2e"])))
        return _rcp(F(1) + _exp2(y))
    e = _exp2(F(F(F(-0.5) * k["kLog2e"] * x) * x))
    t = _rcp(_fma(np.abs(x), scale, F(1)))
    r = np.full_like(x, poly[0])
    for c in poly[1:]:
        r = _fma(r, t.astype(np.float64), c)
    below = F(e * F(t * r))
    return np.where(x > 0, F(1) - below, below)


def _true(x, name):
    t = torch.from_numpy(x.astype(np.float64))
    if name == "silu":
        return torch.sigmoid(t).numpy()
    if name == "gelu":
        return (0.5 * torch.erfc(-t / 2 ** 0.5)).numpy()
    return torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (t + 0.044715 * t ** 3)).numpy()


def _bound(x, name):
    a = np.abs(x.astype(np.float64))
    if name == "silu":
        return 2.0 ** -20 + 1.6 * a * U
    if name == "gelu":
        return 2.0 ** -19 + 1.4 * a * a * U
    return 2.0 ** -20 + 4 * (1.6 * a + 0.072 * a ** 3) * U


@pytest.mark.parametrize("name,most", [("silu", 87.0), ("gelu", 13.0), ("gelu_tanh", 9.8)])  # powers that are normal numbers
def test_factors(name, most):
    x = np.concatenate([np.linspace(-most, most, 400001), np.linspace(-1, 1, 50001), np.logspace(-30, 0, 1001)]).astype(F)
    ref = _true(x, name)
    err = np.abs(_factor(x, name).astype(np.float64) - ref) / ref + 2.0 ** -22 + 2.0 ** -23
    assert (err <= _bound(x, name)).all(), float((err / _bound(x, name)).max())


@pytest.mark.parametrize("name", ACTS)
def test_the_bound_that_the_gpu_tests_use(name):
    """gated_util.act_error is wider than the factor's bound and the rounding of x times it."""
    g = np.linspace(-30, 30, 60001)
    assert (act_error(g) >= _bound(g, name) + 2 * U).all()
