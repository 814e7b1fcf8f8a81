"""The tanh GELU's slope to the last digits of fp32, where its parts cancel.

With z = 2 sqrt(2/pi) (x + 0.044715 x^3), s = 1 / (1 + e^-z), t = 1 - s, a = x s
and z' = dz/dx the slope is s + a t z'.  The bound counts roundings (U = 2^-24):
e^-z is off by a relative E = (4 |z| + 2) U (its argument carries four, the
exponential is within 1 ulp), s by t E + 3 U, t by s E + 4 U if it is taken
without cancellation, a by t E + 4 U and z' by 3 U, so that a t z' is off by E +
12 U with its own product; the last step rounds once.  A t that is taken as the
rounded 1 - s is off by U absolutely, |a| z' U in the slope: 33 U at x = 5, where
the bound is 4 U."""
import math

import pytest
import torch

import act_ref as R
from act_util import rand
from fp4_quantization_block_amd import mx
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _slope(x):
    """act'(x) in 64 bits and the bound."""
    k = 2 * math.sqrt(2 / math.pi)
    z, dz = k * (x + 0.044715 * x ** 3), k * (1 + 3 * 0.044715 * x * x)
    s, t = torch.special.expit(z), torch.special.expit(-z)
    d = s + x * s * t * dz
    e = 4 * z.abs() + 2
    return d, R.U * (s * (t * e + 3) + (x * s).abs() * t * dz * (e + 12) + d.abs()) + R.TINY


@pytest.mark.parametrize("lo,hi", [(-12.0, 12.0), (3.0, 6.0), (-0.5, 0.5), (-110.0, 110.0)])
@pytest.mark.parametrize("cols", [2048, 2051])
def test_tanh_slope(lo, hi, cols):
    """dh = up = 1: dgate is the slope itself."""
    x = torch.linspace(lo, hi, 31 * cols, dtype=torch.float64).float().reshape(31, cols)
    one = torch.ones(31, cols, device=DEV)
    got = mx.mx_glu_backward(one, x.to(DEV), one, "gelu_tanh").dgate
    d, err = _slope(x.double())
    R.within(got, d, err, f"slope on {lo}..{hi}")


def test_tanh_gradient_on_activations():
    """dh up act'(gate) of ordinary activations: two more products."""
    g, u, dh = (rand(k, 257, 2731, scale=s).float() for k, s in ((1, 1.5), (2, 1.5), (3, 1e-3)))
    got = mx.mx_glu_backward(dh.to(DEV), g.to(DEV), u.to(DEV), "gelu_tanh").dgate
    d, err = _slope(g.double())
    f = dh.double() * u.double()
    R.within(got, f * d, f.abs() * err + 2 * R.U * (f * d).abs(), "dgate")
