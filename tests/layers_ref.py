"""Plain 64-bit implementations of the gated block, the layer norm and norms
over many tensors (numpy), and the error bounds the tests hold the library to,
counted in roundings as in ops_ref.py."""
import numpy as np

import ops_ref as ref
from ops_ref import U

# ---- layer norm ------------------------------------------------------------------------------
#
# On the float32 S that the call stores: the mean is float64's, so d = S - m is
# off by the roundings of (S - hi) and of (... - lo), 3 U of it, and by the
# 2^-48 of m that two float32 parts leave.  A thread adds at most 32 squares (7 U
# each, and 32 U of their sum); threads are added in float64.  So the variance
# is off by 40 U at most, r by 20 U and its rounding.
VAR_ERR = 40 * U


def layernorm(s, w, b, eps):
    """(y, bound of y) of float64 s."""
    m = s.mean(1, keepdims=True)
    d = s - m
    r = 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    g = 1.0 if w is None else w
    hw = d * r * g
    y = hw + (0.0 if b is None else b)
    t = np.abs(hw) * (VAR_ERR / 2 + 3 * U + 4 * U) + 2 * U * np.abs(y) + np.abs(r * g * m) * 2.0 ** -46
    return y, t + 1e-37


def layernorm_grad(dy, s, w, eps, ds=None):
    """(dx, dw, db, bounds of each)."""
    rows, D = s.shape
    m = s.mean(1, keepdims=True)
    d = s - m
    r = 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    h = d * r
    g = dy * (1.0 if w is None else w)
    mg = g.mean(1, keepdims=True)
    mgd = (g * d).mean(1, keepdims=True)
    dx = r * (g - mg) - d * (r ** 3 * mgd)
    # sums over a row: a thread's 16, the wave's 6 and the workgroup's 16 additions
    chain = 40 * U
    rho = (chain + 8 * U) / 2 + 4 * U  # r
    far = np.abs(m) * 2.0 ** -46       # what d may be off by besides 3 U of it
    t_mg = (chain + 3 * U) * np.abs(g).mean(1, keepdims=True)
    t_c = r ** 3 * ((chain + 8 * U) * np.abs(g * d).mean(1, keepdims=True) + (3 * rho + 5 * U) * np.abs(mgd) +
                    np.abs(g).mean(1, keepdims=True) * far)
    t = r * (np.abs(g - mg) * (rho + 3 * U) + U * np.abs(g) + t_mg) + np.abs(d) * t_c + \
        (np.abs(d) * 5 * U + far) * np.abs(r ** 3 * mgd) + 2 * U * np.abs(dx)
    if ds is not None:
        dx = dx + ds
        t = t + U * np.abs(dx)
    term = dy * h
    tw = np.abs(term).sum(0) * ((rows + 3) * U + rho + 5 * U) + (np.abs(dy) * r * far).sum(0)
    return dx, term.sum(0), dy.sum(0), t + 1e-37, tw + 1e-37, np.abs(dy).sum(0) * (rows + 3) * U + 1e-37


# ---- norms over many tensors -------------------------------------------------------------------

def clip(tensors, max_norm, eps):
    """(norm, factor): float64 sums leave nothing but the rounding of each."""
    n = np.sqrt(sum(float((x.astype(np.float64) ** 2).sum()) for x in tensors))
    with np.errstate(divide="ignore"):
        f = np.float64(max_norm) / (n + eps) if n + eps > 0 else np.inf
    return n, min(1.0, f) if not np.isnan(f) else f


# ---- the gated block ------------------------------------------------------------------------------

def gated(A, Bg, Bu, K, bias_gate=None, bias_up=None, activation="silu"):
    """(Y, G, U, bounds of each) of float64 operands (K x N weights): the two
    products' bounds of ops_ref.product, the activation's, and the product of
    the two values."""
    G, _, tg, _ = ref.product(A, Bg, K, 1.0, bias_gate)
    U_, _, tu, _ = ref.product(A, Bu, K, 1.0, bias_up)
    a = ref.act(G, activation)
    ta = ref.LIPSCHITZ * tg + (ref.ACT_ERR * np.abs(G) if activation != "none" else 0)
    Y = a * U_
    return Y, G, U_, np.abs(U_) * ta + (np.abs(a) + ta) * tu + 2 * U * np.abs(Y) + 1e-37, tg, tu


def gated_grad(dy, G, U_, activation):
    """(dG, dU, their column sums, bounds of the four)."""
    s, a = ref.slope(G, activation), ref.act(G, activation)
    dg, du = dy * U_ * s, dy * a
    none = activation == "none"
    tg = np.abs(dy * U_) * (0 if none else ref.SLOPE_ERR) + 2 * U * np.abs(dg) + 1e-37
    tu = np.abs(dy) * np.abs(G) * (0 if none else ref.ACT_ERR) + U * np.abs(du) + 1e-37
    n = (dy.shape[0] + 1) * U
    return (dg, du, dg.sum(0), du.sum(0), tg, tu, tg.sum(0) + n * np.abs(dg).sum(0) + 1e-37,
            tu.sum(0) + n * np.abs(du).sum(0) + 1e-37)


def gated_backward(dy, A, Bg, Bu, G, U_, activation):
    """(dA, dBg, dBu, bounds of each) of float64 operands (K x N weights)."""
    dg, du, _, _, tg, tu, _, _ = gated_grad(dy, G, U_, activation)
    M, N = dy.shape

    def prod(x, y, n, tx):
        """x @ y, x off by tx, sums of n float32 terms."""
        return x @ y, (n + 3) * U * (np.abs(x) @ np.abs(y)) + tx @ np.abs(y)
    a, ta = prod(dg, Bg.T, 2 * N, tg)
    b, tb = prod(du, Bu.T, 2 * N, tu)
    dA = a + b
    (x, tx), (y, ty) = prod(dg.T, A, M, tg.T), prod(du.T, A, M, tu.T)
    return dA, x.T, y.T, ta + tb + U * np.abs(dA) + 1e-37, tx.T + 1e-37, ty.T + 1e-37
