"""Activations and their slopes at infinities and in the tails, where a value is
far smaller than its argument.

Tolerances of the tails, relative to the value (a slope: to each of its two
terms) in units of 2^-24.  With x the logistic's argument (z for silu, 2 u for
gelu): the exponent in base 2 is one product for silu (constant and product: 1.25
units) and a cubic for gelu (constants, square, fma and product: 6 units), each
worth |x| of the power; ex2 and reciprocal approximations, 1 + e and the last
product: 4 + 2 + 1 + 1.  A slope's second term holds the logistic twice and four
more factors.  1e-35 absolute: results below that are not told apart.
"""
import numpy as np
import pytest
import torch

from all_mxfp8_block_gb300 import mxa2a
from tests import operators_ref as R
from tests.test_gpu_linear import ACT
from tests.test_gpu_moe import TYPE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_slope_at_infinities(act):
    # the slopes' limits: 1 at +inf, 0 at -inf; a NaN stays one
    inf = float("inf")
    z = torch.tensor([inf, -inf, float("nan"), 3e38, -3e38] + [1.0] * 27).bfloat16().cuda()[None]
    one = torch.ones(1, 32, dtype=torch.bfloat16, device="cuda")
    l = mxa2a.Linear(1, 1, 32, 32, training=True)
    db = torch.full((1, 32), 7.0, device="cuda")
    l.backward(1, one, z, ACT[act], TYPE["e4m3"], None, None, None, None, None, None, 0, db)
    got = R.f64(db)[0]
    assert np.isnan(got[2])
    assert np.abs(got[[0, 1, 3, 4]] - [1, 0, 1, 0]).max() <= 1e-6, got[:5]


U = 2.0 ** -24


def argument(z, act):
    """x, its derivative, and the units that one |x| costs."""
    if act == "silu":
        return z, np.ones_like(z), 1.25
    a, b = 2 * np.sqrt(2 / np.pi), 0.044715
    return a * (z + b * z ** 3), a * (1 + 3 * b * z * z), 6.0


@pytest.mark.parametrize("act,low,high", [("silu", -86.0, 86.0), ("gelu", -9.9, 30.0), ("silu", -1.0, 1.0), ("gelu", -1.0, 1.0)])
def test_values_in_the_tails(act, low, high):
    # no tokens' sums: the value before the activation is the bias, to the bit
    N = 4096
    bias = torch.linspace(low, high, N).cuda()[None]
    zeros = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    out = torch.full((1, N), 7.0, device="cuda")
    l = mxa2a.Linear(1, 1, N, 32)
    l.run(1, zeros(1, 32), zeros(1, 1, 512), zeros(N, 32), zeros(1, N // 128, 512), out, TYPE["f32"], bias=bias, activation=ACT[act])
    z = R.f64(bias)
    x, _, units = argument(z, act)
    ref = z / (1 + np.exp(-x))
    R.check(out, ref, (units * np.abs(x) + 8) * U * np.abs(ref) + 1e-35)


@pytest.mark.parametrize("act,low,high", [("silu", -86.0, 86.0), ("gelu", -9.9, 9.9), ("silu", -4.0, 4.0), ("gelu", -4.0, 4.0)])
def test_slopes_in_the_tails(act, low, high):
    # one token with dy = 1: dbias is the slope
    N = 2048
    zb = torch.linspace(low, high, N).bfloat16().cuda()[None]
    db = torch.zeros(1, N, device="cuda")
    l = mxa2a.Linear(1, 1, N, 32, training=True)
    l.backward(1, torch.ones(1, N, dtype=torch.bfloat16, device="cuda"), zb, ACT[act], TYPE["e4m3"], None, None, None, None, None, None, 0, db)
    z = R.f64(zb)
    x, dx, units = argument(z, act)
    s, rest = 1 / (1 + np.exp(-x)), 1 / (1 + np.exp(x))
    first, second = s, z * s * rest * dx
    one = units * np.abs(x) + 8
    R.check(db, first + second, (one * first + (2 * one + 12) * np.abs(second) + np.abs(first + second)) * U + 1e-35)
