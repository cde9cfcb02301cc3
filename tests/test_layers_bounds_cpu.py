"""The bounds of layers_bounds.py on the host: the kernels' arithmetic stays
inside them, and what they are there to catch does not."""
import numpy as np
import pytest

import layers_bounds as bounds
import layers_ref
from layers_bounds import planted, rows_of


@pytest.mark.parametrize("D", [5, 700, 3000, 20003])
def test_kernel_arithmetic_is_within(D):
    rng = np.random.default_rng(1)
    s = rows_of(D)
    dy, w, b = (rng.standard_normal(n).astype(np.float32) for n in ((10, D), D, D))
    f = lambda v: v.astype(np.float64)  # noqa: E731
    eps = float(np.float32(1e-5))
    y, t = bounds.forward(f(s), f(w), f(b), eps)
    assert (np.abs(bounds.kernel_forward(s, w, b, eps) - y) <= t).all()
    dx, _, _, t, _, _ = bounds.backward(f(dy), f(s), f(w), eps)
    off = np.abs(bounds.kernel_backward(dy, s, w, eps) - dx) / t
    assert off.max() <= 1, off.max(1)
    # the factor of d on its own leaves float32
    off = np.abs(bounds.kernel_backward(dy, s, w, eps, cube=True) - dx) / t
    assert (off[4:8].max(1) > 10).all(), off.max(1)
    small = (s[:1] * np.float32(1e-21))
    dx, _, _, t, _, _ = bounds.backward(f(dy[:1]), f(small), f(w), 0.0)
    assert (np.abs(bounds.kernel_backward(dy[:1], small, w, 0.0) - dx) <= t).all()
    assert not np.isfinite(bounds.kernel_backward(dy[:1], small, w, 0.0, cube=True)).all()


@pytest.mark.parametrize("D", [64, 700, 2052, 20004])
def test_row_sums_in_float32_are_outside(D):
    s, t, dy = planted(D)
    f = lambda v: v.astype(np.float64)  # noqa: E731
    y, ty = bounds.forward(f(s), None, None, 0.0)
    assert (np.abs(bounds.kernel_forward(s, None, None, 0.0) - y) <= ty).all()
    assert (np.abs(bounds.kernel_forward(s, None, None, 0.0, np.float32) - y) > ty).any()
    dx, _, _, tx, _, _ = bounds.backward(f(dy), f(t), None, 0.0)
    assert (np.abs(bounds.kernel_backward(dy, t, None, 0.0) - dx) <= tx).all()
    assert (np.abs(bounds.kernel_backward(dy, t, None, 0.0, np.float32) - dx) > tx).any()


def test_the_two_references_agree():
    rng = np.random.default_rng(2)
    s, dy, ds = (rng.standard_normal((6, 40)) for _ in range(3))
    w, b = rng.standard_normal(40), rng.standard_normal(40)
    assert np.allclose(bounds.forward(s, w, b, 1e-3)[0], layers_ref.layernorm(s, w, b, 1e-3)[0], rtol=0, atol=1e-13)
    for x, y in zip(bounds.backward(dy, s, w, 1e-3, ds)[:3], layers_ref.layernorm_grad(dy, s, w, 1e-3, ds)[:3]):
        assert np.allclose(x, y, rtol=0, atol=1e-12)
