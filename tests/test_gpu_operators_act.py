"""Activations and their slopes over their whole range, in binary32, against
binary64: the digits of the negative tail, not only its size.  Bounds count
roundings: u = 2^-24 an operation, 4 u for 2^x, 2 u for a reciprocal."""
import numpy as np
import pytest
import torch

import bit_fwht_hadamard_b200 as q
import operators_ref as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = 2.0 ** -120                                           # results below this may be flushed to zero
# E = e^-|x| (e^(-z^2/2) for GELU) may be flushed below 2^-126.  For a slope that is f (1 + z g x'), f, g <= 1, it takes
# 2^-126 (1 + |z| x') with it: up to 2^-118 for the tanh form, whose x' is 23 at z = -10, where E = 2^-126.
ACT = {n: i for i, n in enumerate(R.ACTS)}


def grid():
    """From -13 to 13, and from 1e-6 to 1 on both sides."""
    a = torch.linspace(-13, 13, 1 << 17, dtype=torch.float64)
    b = torch.logspace(-6, 0, 1 << 14, dtype=torch.float64)
    return torch.cat([a, b, -b]).float().cuda()


def parts(z, name):
    """(act, slope, relative error of the tail factor in u, the terms' sizes, what a
    flushed E takes of the slope): the sigmoid or normal distribution function
    behind each, without cancellation."""
    if name == "gelu":
        # Phi(-a) = E m(a): E = 2^y, y = -a^2/2 log2 e after two roundings and a rounded constant, (4 + 1.05 a^2) u;
        # m = N(a) / D(a), positive terms of degree 3 and 4: the quotient's own fit (1.1 + 0.43 a^2) u, a rounding a
        # step and the coefficients' (4 u and 5 u), two for the reciprocal, one for the product; two more products
        phi = 0.5 * torch.special.erfc(-z / 2 ** 0.5)
        pdf = torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5
        e = 1.48 * z * z + 19.1
        small = 0.5 * torch.special.erfc(z.abs() / 2 ** 0.5)
        return z * phi, phi + z * pdf, e, (z * small).abs(), small + z.abs() * pdf, TINY
    if name == "silu":
        # the exponent to both its words: 2^x 4 u, correction 2 u, 1 + E, reciprocal 2 u, two products
        x, dx, e = z, torch.ones_like(z), torch.full_like(z, 12.0)
    else:
        # x = 2 sqrt(2/pi) (z + 0.044715 z^3): four roundings and two constants, 5 |x| u of E
        c = 2 * (2 / np.pi) ** 0.5
        x, dx = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)
        e = 12 + 5 * x.abs()
    f, g = torch.sigmoid(x), torch.sigmoid(-x)
    small = torch.minimum(f, g)
    # f itself rounds as the tail where it is the small one, and to 4 u where it is near one
    flushed = 2.0 ** -126 * (1 + z.abs() * dx)
    return z * f, f + z * f * g * dx, e, (z * small).abs(), small + z.abs() * f * g * dx, flushed


def show(err, bound, z, got, want, name):
    bad = ~(err <= bound)
    if bool(bad.any()):
        r = torch.where(bad, err / bound, torch.zeros_like(err))
        i = int(r.argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {z.numel()} outside; worst at z = {float(z[i])}: got "
                             f"{float(got[i])} want {float(want[i])} bound {float(bound[i])}")


def forward(z, name, dt):
    """act(z) of the library: the epilogue of an empty sum whose bias is z."""
    n = z.numel()
    A, B = R.random_operand(1, 0, q.MXFP4, 1), R.random_operand(n, 0, q.MXFP4, 2)
    return q.gemm_epilogue(A, B, 1, n, 0, q.MXFP4, bias=z, act=ACT[name], out_dtype=dt)[0][0]


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_activation_keeps_the_tail(name):
    z = grid()
    z = z[:z.numel() // 8 * 8]
    want, _, e, tail, _, _ = parts(z.double(), name)
    # the tail's own roundings, and four of the result (GELU's one, the sigmoid near one and its product)
    bound = e * U * tail + 4 * U * torch.where(z > 0, want.abs(), 0 * want) + TINY
    got = forward(z, name, torch.float32).double()
    show((got - want).abs(), bound, z, got, want, name)
    got = forward(z, name, torch.bfloat16).double()
    show((got - want).abs(), bound + 2.0 ** -8 * (1 + 2.0 ** -6) * want.abs(), z, got, want, name + " bf16")


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_slope_keeps_the_tail(name):
    z = grid()
    z = z[:z.numel() // 8 * 8].view(1, -1)
    _, want, e, _, mag, flushed = parts(z.double(), name)
    # the other factors' words and products behind the tail's; six of the result where the sigmoid is near one
    bound = (e + 8) * U * mag + 6 * U * torch.where(z > 0, want.abs(), 0 * want) + flushed
    got, _ = q.epilogue_backward(torch.ones_like(z), z, act=ACT[name])
    show((got.double() - want).abs().view(-1), bound.view(-1), z.view(-1), got.view(-1), want.view(-1), name)
