"""Pins of the gated block's oracle (oracle/mx.py): the activations against their
definitions, and the gradients against differences of the block itself."""

import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import mx

ACTS = ["silu", "gelu", "gelu_tanh"]


def _exp(x):
    """e**x of a Fraction, by its series after halving the argument: 60 terms of a
    number below 1/16 leave less than 2**-200."""
    n = 0
    while abs(x) > Fraction(1, 16):
        x, n = x / 2, n + 1
    s, t = Fraction(1), Fraction(1)
    for i in range(1, 40):
        t = t * x / i
        s += t
    for _ in range(n):
        s = Fraction(int(s * s * (1 << 240)), 1 << 240)
    return s


@pytest.mark.parametrize("g", [-9.5, -3.0, -1.0, -0.125, 0.0, 0.375, 1.0, 2.5, 8.0])
def test_silu_and_gelu_tanh_by_their_definitions(g):
    f = Fraction(g)
    silu = f / (1 + _exp(-f))
    assert mx.activation(g, "silu")[0] == pytest.approx(float(silu), rel=4e-15, abs=1e-300)
    y = Fraction(math.sqrt(2 / math.pi)) * (f + Fraction(0.044715) * f ** 3)
    e = _exp(2 * y)
    tanh = (e - 1) / (e + 1)
    # (1 + tanh cancels below zero: the definition in rational numbers does not)
    assert mx.activation(g, "gelu_tanh")[0] == pytest.approx(float(f * (1 + tanh) / 2), rel=1e-12, abs=1e-300)


@pytest.mark.parametrize("g", [-6.0, -2.0, -0.5, 0.0, 0.25, 1.5, 5.0])
def test_gelu_by_the_normal_distribution(g):
    """Phi(g) as the integral of the density by Simpson's rule from far below."""
    n = 40000
    x = np.linspace(-14.0, g, n + 1)
    f = np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    h = (g + 14.0) / n
    phi = h / 3 * (f[0] + f[-1] + 4 * f[1::2].sum() + 2 * f[2:-1:2].sum())
    assert mx.activation(g, "gelu")[0] == pytest.approx(g * phi, rel=1e-9, abs=1e-15)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    rng = np.random.default_rng(1)
    g, u, dh = rng.standard_normal((3, 200)) * 3
    dg, du = mx.gated_grad(dh, g, u, act)
    e = 1e-5
    num_g = (mx.gated(g + e, u, act) - mx.gated(g - e, u, act)) / (2 * e) * dh
    num_u = (mx.gated(g, u + e, act) - mx.gated(g, u - e, act)) / (2 * e) * dh
    # third derivatives of the activations are below 3: e^2/6 of that, and the differences' rounding
    tol = 1e-9 * (1 + np.abs(dh) * (1 + np.abs(u)) * (1 + np.abs(g)))
    assert (np.abs(dg - num_g) <= tol).all() and (np.abs(du - num_u) <= tol).all()


@pytest.mark.parametrize("act", ACTS)
def test_far_ends(act):
    a, d = mx.activation(np.array([-200.0, -40.0, 40.0, 200.0]), act)
    assert np.allclose(a, [0, 0, 40, 200], atol=1e-14) and np.allclose(d, [0, 0, 1, 1], atol=1e-14)
