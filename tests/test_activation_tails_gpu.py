"""Activations and their slopes in the lower tail, to a relative bound: there
they are products of small factors, and nothing cancels.

The bounds count roundings (U = 2^-24 each, a hardware exponential or
reciprocal two) along the formula in float32:

exponential exp(-t) of an exact t: 2^x, its argument's low part carried, 3 U;
gelu: exp(-z^2 / 2) with the square's rounding carried, 5 U.  t = 1 / (1 + a/2)
  with a = |z| / sqrt 2: constant, sum, reciprocal, 4 U, and exp(a^2) erfc(a) =
  t P(t) moves by up to 2.3 times t's relative error, 9.2 U; P's coefficients,
  their sum and the fit 5.1 U; two products.  Phi 21.3 U, gelu one more.
silu: exponential 3 U, 1 + e and its reciprocal 3 U, two products: 8 U.
gelu_tanh: the exponent 2u = 2c (z + a z^3) has 7 roundings (constants, cube,
  sum, product), which move the sigmoid by |2u| times as much, then as silu.
Slopes sum two terms: each term's bound, a few products, and the sum's U.
"""
import math

import numpy as np
import pytest
import torch
from scipy.special import erfc

import fp32_gemm_sgemm_amd as sg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -126
C = math.sqrt(2 / math.pi)


def tail(name, z):
    """(value, slope, bound of the value, bound of the slope) in 64 bits."""
    if name == "gelu":
        phi, gauss = erfc(-z / math.sqrt(2)) / 2, z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        v, d = z * phi, phi + gauss
        tv, td = 23 * U * np.abs(v), 22 * U * phi + 8 * U * np.abs(gauss) + U * np.abs(d)
    else:
        u2 = z if name == "silu" else 2 * C * (z + 0.044715 * z ** 3)
        du = np.ones_like(z) if name == "silu" else 2 * C * (1 + 3 * 0.044715 * z * z)
        e = np.exp(u2)
        s, rest = e / (1 + e), 1 / (1 + e)
        rel = 8 * U if name == "silu" else (8 + 7 * np.abs(u2)) * U
        v, d = z * s, s + z * s * rest * du
        # (the second term: 1 - sigma, the cubic's slope and the products, 10 U more)
        tv, td = (rel + U) * np.abs(v), rel * s + (rel + 10 * U) * np.abs(z * s * rest * du) + U * np.abs(d)
    # below the smallest normal value a step is 2^-149; exponentials there are 0
    return v, d, tv + 2.0 ** -149, td + 2.0 ** -149


# z down to where the value or the exponential falls below 2^-126
LOWEST = {"gelu": -12.9, "gelu_tanh": -9.9, "silu": -87.0}


@pytest.mark.parametrize("name", LOWEST)
@pytest.mark.parametrize("rows", [1, 300])
def test_lower_tail(name, rows):
    """rows = 1 goes through the kernels of few rows, 300 through the tiles."""
    z = np.linspace(LOWEST[name], -1.0, 20001).astype(np.float32)
    v, d, tv, td = tail(name, z.astype(np.float64))
    assert np.abs(v).min() > TINY
    one, zd = torch.ones(rows, 1, device="cuda"), torch.from_numpy(z).cuda()[None, :].contiguous()
    pre = zd.expand(rows, -1).contiguous()
    got = {"value": (sg.sgemm_epilogue(one, zd, activation=name), v, tv),
           "slope": (sg.sgemm_epilogue(one, torch.ones_like(zd), activation=name, grad_pre=pre), d, td),
           "gradient": (sg.activation_grad(torch.ones_like(pre), pre, name, dbias=False)[0], d, td)}
    torch.cuda.synchronize()
    for what, (t, want, bound) in got.items():
        err = np.abs(t.cpu().double().numpy() - want) / bound
        print(f"{name} {what} rows {rows}: worst {err.max():.3f} of its bound, at z = {z[err.max(0).argmax()]}", flush=True)
        assert err.max() <= 1, f"{name} {what}: {err.max():.2f} times the bound at z = {z[err.max(0).argmax()]}"
