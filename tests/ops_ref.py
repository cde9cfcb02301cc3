"""Plain 64-bit implementations of the operators around a product (numpy), and
the error bounds the tests hold the library to.

Bounds count roundings to nearest: one float32 rounding is off by at most
U = 2^-24 of the value, one e4m3 rounding by 2^-4 of it (or half the smallest
step, 2^-10, near zero).  A sum of n float32 terms, in whatever order, is off
by at most about n * U * (the sum of the terms' magnitudes); where the kernel's
additions are fewer (a tree over threads), the count of the longest chain
stands for n.
"""
import math

import numpy as np
from scipy.special import erf

U = 2.0 ** -24
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
GELU_C = math.sqrt(2 / math.pi)


def sigmoid(t):
    with np.errstate(over="ignore"):  # 1 / inf is the right 0
        return 1 / (1 + np.exp(-t))


def act(z, name):
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "gelu":
        return z * 0.5 * (1 + erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(GELU_C * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * sigmoid(z)
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1 + erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = np.tanh(GELU_C * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_C * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = sigmoid(z)
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


# An activation's value: exponential (2 U), sum, reciprocal (2 U) and products,
# with the argument's own roundings weighted by how far it moves the value, and
# gelu's polynomial (4e-7 of its tail): within 16 U of |z|.  Its slope, at most
# 1.2 in magnitude, sums two such terms: within 32 U.
ACT_ERR = 16 * U
SLOPE_ERR = 32 * U
LIPSCHITZ = 1.2  # the largest slope of any activation


def product(A, B, K, alpha=1.0, bias=None, activation="none", residual=None, grad_pre=None):
    """(C, z, bound of C, bound of z) of an epilogue product of float64 op(A) and
    op(B) (2-D or batches)."""
    s = np.matmul(A, B)
    mag = abs(alpha) * np.matmul(np.abs(A), np.abs(B))
    z = alpha * s
    tz = (K + 3) * U * mag
    if bias is not None:
        z = z + bias
        tz = tz + U * (np.abs(z) + np.abs(bias))
    if grad_pre is not None:
        g = slope(grad_pre, activation)
        y = z * g
        ty = LIPSCHITZ * tz + SLOPE_ERR * np.abs(z) + U * np.abs(y)
    else:
        y = act(z, activation)
        ty = LIPSCHITZ * tz + (ACT_ERR * np.abs(z) if activation != "none" else 0)
    if residual is not None:
        y = y + residual
        ty = ty + U * np.abs(y)
    return y, z, ty + 1e-37, tz + 1e-37


def chain(D):
    """Longest chain of additions over a row of D values: a thread's own (16 up
    to 16384 values, then its share of 1024 threads), the shuffles and the waves."""
    return (16 if D <= 16384 else 4 * math.ceil(D / 4096)) + 6 + 16


def rmsnorm(x, w, eps, residual=None):
    """(y, s, bound of y, relative bound of 1/rms)."""
    s = x if residual is None else x + residual
    D = x.shape[1]
    r = 1 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    y = s * r * (1 if w is None else w)
    # the squares' roundings and S's own (twice), their sum, mean, eps, root, reciprocal
    rho = (chain(D) + 4) / 2 * U + 4 * U
    return y, s, np.abs(y) * (rho + 4 * U) + 1e-37, rho


def e4m3_values():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 8 * 2.0 ** -6)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


E4M3 = e4m3_values()


def check_codes(q, scale, y, ty, rel_scale):
    """8-bit rows against the values they stand for: the scale within its own
    bound, and each value off by at most half a step beyond the value's bound."""
    want = np.maximum(np.abs(y).max(1) / 448, 2.0 ** -126)
    # (the row's largest value carries its own error into the scale)
    t = np.abs(ty).max(1) / 448 + want * (rel_scale + 3 * U)
    assert np.all(np.abs(scale - want) <= t), np.max(np.abs(scale - want) / want)
    deq = q * scale[:, None]
    # y * (1 / scale): two roundings before the code's own
    half = np.maximum(np.abs(y) * 2.0 ** -4 * (1 + 8 * U), scale[:, None] * 2.0 ** -10)
    err = np.abs(deq - y)
    bad = err > half + ty + np.abs(y) * 4 * U
    assert not bad.any(), (int(bad.sum()), float((err / half)[bad].max()))


def rmsnorm_grad(dy, s, w, eps, ds=None):
    """(dx, dw, bound of dx, bound of dw)."""
    rows, D = s.shape
    r = 1 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    rho = (chain(D) + 4) / 2 * U + 4 * U
    g = dy * (1 if w is None else w)
    dot = (g * s).sum(1, keepdims=True)
    mag = np.abs(g * s).sum(1, keepdims=True)
    c = r ** 3 * dot / D
    dx = r * g - s * c
    tc = r ** 3 / D * ((chain(D) + 4) * U * mag + (3 * rho + 5 * U) * np.abs(dot))
    t = np.abs(r * g) * (rho + 3 * U) + np.abs(s) * tc + np.abs(s * c) * 2 * U + 2 * U * np.abs(dx)
    if ds is not None:
        dx = dx + ds
        t = t + U * np.abs(dx)
    term = dy * s * r
    return dx, term.sum(0), t + 1e-37, np.abs(term).sum(0) * ((rows + 3) * U + rho) + 1e-37


def act_grad(dy, z, name):
    """(dz, dbias, bound of dz, bound of dbias)."""
    dz = dy * (slope(z, name) if name != "none" else 1.0)
    t = np.abs(dy) * SLOPE_ERR + U * np.abs(dz) if name != "none" else np.zeros_like(dz)
    return dz, dz.sum(0), t + 1e-37, t.sum(0) + np.abs(dz).sum(0) * (dy.shape[0] + 1) * U + 1e-37


def within(got, want, bound, what=""):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.nanmax(err / bound):.3g} bounds"
