"""GPU parity of the activations themselves, relative to their value: also far below zero, where it is small.

A layer with the identity as its weights hands each activation its argument exactly.  u = 2^-24.  Bounds of fp32, by
counting roundings: the exponential within 2^-22 of itself (1 ulp of the hardware's, two more roundings), 1 + e one
rounding, the reciprocal 1 ulp, the product one: 2^-21 together.  The tanh GELU's argument a has seven roundings on the
way: 7 u |a| < 2^-21 |a| more.  Slopes add terms of the size of p and |z| p, each with such an error.
"""
import math

import pytest
import torch

import convolution_forward_conv2d_amd as mic
import feed_forward_ref as R
from test_feed_forward_gpu import BF16, F32, dev

pytestmark = pytest.mark.gpu

N = 64


def applied(z, name, dtype):
    """(value, slope) of the activation at z, on rows enough for a layer's tiles and on a single one."""
    rows = z.to(dtype).to(dev()).reshape(-1, N)
    eye = torch.eye(N, device=dev()).to(dtype)
    y = mic.linear(rows, eye, activation=name)
    assert torch.equal(mic.linear(rows[:1], eye, activation=name), y[:1])
    dx, _, _ = mic.linear_backward(torch.ones_like(rows), rows, eye, preact=rows, activation=name)
    return R.d(rows), R.d(y), R.d(dx)


def argument(z, name):
    return z if name == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)


def holds(got, want, bound, z):
    over = (got - want).abs() - bound
    i = int(over.argmax())
    at = [float(t.reshape(-1)[i]) for t in (z, got, want, bound)]
    assert float(over.max()) <= 0, "at %.9g: %.9g, expected %.9g +- %.3g" % tuple(at)


@pytest.mark.parametrize("name,low", [("silu", 85.0), ("gelu_tanh", 9.0)])
def test_fp32_is_as_exact_far_from_zero(name, low):
    z, y, slope = applied(torch.linspace(-low, low, 64 * N, dtype=torch.float64), name, F32)
    a = argument(z, name)
    e = 2.0 ** -21 * (1 + (a.abs() if name == "gelu_tanh" else 0))
    want = z * torch.sigmoid(a)
    holds(y, want, e * want.abs() + 1e-36, z)
    p, rise = torch.sigmoid(a), 1 if name == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    # p, then z p (1 - p) a': of its factors p is off by e, 1 - p by e p + u, the rest by roundings
    holds(slope, p + z * p * (1 - p) * rise, e * p + z.abs() * p * rise * (2 * e + 2.0 ** -21) + 1e-36, z)


def test_bf16_gelu_keeps_its_precision_far_below_zero():
    """The tail is within 2^-14 of itself, its exponential's argument within 2^-23 z^2, the output rounds to 2^-8."""
    z, y, slope = applied(-torch.logspace(-3, math.log10(12.9), 64 * N, dtype=torch.float64), "gelu", BF16)
    tail = 0.5 * torch.erfc(-z / math.sqrt(2))
    e = 2.0 ** -14 + 2.0 ** -23 * z * z + 2.0 ** -21
    holds(y, z * tail, (2.0 ** -8 * (1 + e) + e) * (z * tail).abs() + 1e-38, z)
    bell = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    want = tail + z * bell
    # dz rounds to bf16, the product with the identity is exact, and so is its rounding
    holds(slope, want, 2.0 ** -8 * want.abs() + 1.01 * e * (tail + z.abs() * bell) + 1e-38, z)
