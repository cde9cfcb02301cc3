"""Error bounds of the float32 layer norm and its gradient, counted from what
the kernels round, and the kernels' arithmetic in numpy.

Row sums are float64: of a row's D values they leave at most a few hundred times
2^-53 of the sum of magnitudes, and the variance from sums about the first value
D times that (the first value itself adds (m - x0)^2 / D to the variance).  SUM
stands for both, up to D = 2^15.  What else is rounded:

  hi + lo      the mean in two float32 parts, 2^-48 of it
  d            s - hi and (s - hi) - lo: 2 U of d, and U of lo (2^-48 of the mean)
  r            U
  h = d r      U
  y            one fused multiplication and addition, U of y
  g = dY w     U of g where there is a w, in the row sums of g and g h too
  mg, p        the means of g and g h: U of each
  dX           g - mg, h p, their difference, its product with r: U of each

A float32 result below 2^-126 is off by half of 2^-149 instead.
"""
import numpy as np

U = 2.0 ** -24
SUM = 2.0 ** -30
FAR = 2.0 ** -46
TINY = 1e-44


def _row(s, eps):
    m = s.mean(1, keepdims=True)
    d = s - m
    r = 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    return m, d, r


def forward(s, w, b, eps):
    """(y, bound) of float64 rows."""
    m, d, r = _row(s, eps)
    g = 1.0 if w is None else w
    hw = d * r * g
    y = hw + (0.0 if b is None else b)
    return y, np.abs(hw) * (4 * U + SUM) + np.abs(r * g * m) * FAR + U * np.abs(y) + TINY * (1 + np.abs(g))


def backward(dy, s, w, eps, ds=None):
    """(dx, dw, db, bounds of each) of float64 rows."""
    rows, D = s.shape
    m, d, r = _row(s, eps)
    h = d * r
    far = np.abs(r * m) * FAR
    th = np.abs(h) * (4 * U + SUM) + far
    g, tg = (dy, 0.0 * dy) if w is None else (dy * w, U * np.abs(dy * w))
    mg, p = g.mean(1, keepdims=True), (g * h).mean(1, keepdims=True)
    size = np.abs(g).mean(1, keepdims=True)
    # (sums of g (s - x0): |s - x0| r is sqrt(D) at most beside |h|)
    t_mg = tg.mean(1, keepdims=True) + U * np.abs(mg) + SUM * 2.0 ** -16 * size
    t_p = (tg * np.abs(h)).mean(1, keepdims=True) + (U + SUM) * np.abs(p) + SUM * 2.0 ** -14 * size * np.sqrt(D)
    a, c = g - mg, h * p
    dx = r * (a - c)
    t = r * (tg + t_mg + U * np.abs(a) + np.abs(h) * t_p + np.abs(p) * th + U * np.abs(c) + TINY) + \
        (3 * U + SUM) * np.abs(dx)
    if ds is not None:
        dx = dx + ds
        t = t + U * np.abs(dx)
    term = dy * h
    tw = (np.abs(dy) * th).sum(0) + np.abs(term).sum(0) * (rows + 8) * U
    return dx, term.sum(0), dy.sum(0), t + TINY, tw + TINY, np.abs(dy).sum(0) * (rows + 8) * U + TINY


# ---- the kernels' arithmetic ------------------------------------------------------------------------

F = np.float32


def row_sum(x):
    """Rows added one value after the other in x's type, as a thread adds its own."""
    return np.cumsum(x, axis=1, dtype=x.dtype)[:, -1:].astype(np.float64)


def moments(s, eps, acc=np.float64):
    """(hi, lo, r in float64, e's mean, e) of float32 rows, sums in `acc`."""
    D = s.shape[1]
    x0 = s[:, :1].astype(acc)
    e = s.astype(acc) - x0
    me = row_sum(e) / D
    var = row_sum(e * e) / D - me * me
    with np.errstate(divide="ignore"):
        rd = 1 / np.sqrt(np.maximum(var, 0.0) + float(F(eps)))
    m = x0.astype(np.float64) + me
    hi = m.astype(F)
    return hi, (m - hi).astype(F), rd, me, e


def kernel_forward(s, w, b, eps, acc=np.float64):
    hi, lo, rd, _, _ = moments(s, eps, acc)
    h = ((s - hi) - lo) * rd.astype(F)
    return (h.astype(np.float64) * (1 if w is None else w) + (0 if b is None else b)).astype(F)


def kernel_backward(dy, s, w, eps, acc=np.float64, cube=False):
    """dX.  cube: by mean(g d) r^3 in float32 instead of mean(g h)."""
    hi, lo, rd, me, e = moments(s, eps, acc)
    g = dy if w is None else dy * w
    D = s.shape[1]
    q2, q3 = row_sum(g.astype(acc)), row_sum(g.astype(acc) * e)
    d, r, mg = (s - hi) - lo, rd.astype(F), (q2 / D).astype(F)
    with np.errstate(over="ignore", invalid="ignore"):
        if cube:
            return r * (g - mg) - d * ((q3 - me * q2) / D * rd ** 3).astype(F)
        return r * ((g - mg) - (d * r) * ((q3 - me * q2) / D * rd).astype(F))


# ---- rows that show them --------------------------------------------------------------------------

def rows_of(D, seed=0):
    """Rows of every size whose spread and its inverse are normal float32."""
    x = np.random.default_rng(seed).standard_normal((10, D))
    scale = np.array([1, 1e15, 1e19, 1e20, 1e22, 1e24, 1e30, 1e36, 1e-3, 1])[:, None]
    x = (x * scale).astype(np.float32)
    x[8] += np.float32(1e6)
    x[9] = 0
    x[9, 0] = -1e30
    return x


def planted(D):
    """(s, dy): rows whose sums, of s and s^2, of g and g h, need more than
    float32: large values that cancel beside ones that count."""
    big = 2.0 ** 26
    s = np.tile([big, 1, 1, -big], D // 4).astype(np.float32)[None, :]
    t = np.tile([-1, 1, 2, -1], D // 4).astype(np.float32)[None, :]
    return s, t, np.tile([big, 1, 3, -big], D // 4).astype(np.float32)[None, :]
