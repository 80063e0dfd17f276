"""The norm's and SwiGLU's oracle: values by hand, gradients against differences."""

import numpy as np

from oracle import norm
from oracle.swiglu import swiglu


def _bits(v):
    return (np.asarray(v, np.float32).view(np.uint32) >> 16).astype(np.uint16)   # exact values only


def test_by_hand():
    s = np.array([[3.0, -4.0, 0.0, 0.0]])
    rstd, y = norm.rms_norm(s, np.array([1.0, 0.5, 1.0, 2.0]), 0.25)
    np.testing.assert_allclose(rstd, [1 / np.sqrt(6.5)])          # 25 / 4 + 0.25
    np.testing.assert_allclose(y, [[3 / np.sqrt(6.5), -2 / np.sqrt(6.5), 0, 0]])


def test_sum_is_rounded_once():
    # 256 + 0.5 and 256 + 1 lie between BF16's 256 and 258: the tie goes to the even 256
    got = norm.residual_sum(_bits([256.0, 256.0, 256.0, -3.0]), _bits([0.5, 1.0, 1.5, 3.0]))
    np.testing.assert_array_equal(got, [256.0, 256.0, 258.0, 0.0])


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(0)
    s, w, ds = rng.normal(size=(5, 32)), rng.normal(size=32), rng.normal(size=(5, 32))
    dy, eps, h = rng.normal(size=(5, 32)), 1e-3, 1e-6
    rstd, _ = norm.rms_norm(s, w, eps)
    dx, dw = norm.rms_norm_backward(dy, s, rstd, w, ds)
    f = lambda s, w: (norm.rms_norm(s, w, eps)[1] * dy).sum() + (s * ds).sum()
    for _ in range(8):
        a, b = rng.normal(size=s.shape), rng.normal(size=w.shape)
        num = (f(s + h * a, w) - f(s - h * a, w)) / (2 * h)
        np.testing.assert_allclose((dx * a).sum(), num, rtol=1e-6, atol=1e-7)
        num = (f(s, w + h * b) - f(s, w - h * b)) / (2 * h)
        np.testing.assert_allclose((dw * b).sum(), num, rtol=1e-6, atol=1e-7)


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(1)
    g, u, dh, h = rng.normal(size=400) * 4, rng.normal(size=400), rng.normal(size=400), 1e-6
    dg, du = norm.swiglu_backward(dh, g, u)
    np.testing.assert_allclose(dg, dh * (swiglu(g + h, u) - swiglu(g - h, u)) / (2 * h), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(du, dh * (swiglu(g, u + h) - swiglu(g, u - h)) / (2 * h), rtol=1e-6, atol=1e-8)


def test_swiglu_gradient_at_the_ends():
    dg, du = norm.swiglu_backward(np.ones(4), np.array([0.0, 800.0, -800.0, -0.0]), np.full(4, 2.0))
    np.testing.assert_array_equal(dg, [1.0, 2.0, 0.0, 1.0])
    np.testing.assert_array_equal(du, [0.0, 800.0, 0.0, 0.0])
