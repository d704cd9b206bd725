"""Pins of oracle/layer.py: gradients against differences of the function, the
functions against closed forms, and the reach of codes against planted mistakes."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import layer, quant

EPS = 1e-6


def rng(seed=0):
    return np.random.default_rng(seed)


def difference(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_rmsnorm_closed_forms():
    y, rstd = layer.rmsnorm(np.array([[3.0, -3.0], [0.0, 0.0]]), np.array([1.0, 2.0]), 16.0)
    assert np.allclose(rstd, [1 / 5, 1 / 4]) and np.allclose(y, [[0.6, -1.2], [0.0, 0.0]])
    r = rng().standard_normal((4, 64))
    y, _ = layer.rmsnorm(r, np.ones(64), 1e-300)
    assert np.allclose(np.mean(y * y, axis=1), 1.0)
    assert np.allclose(layer.rmsnorm(1024.0 * r, np.ones(64), 1e-300)[0], y)


@pytest.mark.parametrize("cols", [1, 2, 7, 130])
def test_rmsnorm_backward_is_the_derivative(cols):
    g = rng(cols)
    r, w, dy, dsum, d = (g.standard_normal((5, cols)) for _ in range(5))
    w = w[0]
    dx, dw = layer.rmsnorm_backward(dy, r, w, 0.1, dsum)
    f = lambda r: np.sum(dy * layer.rmsnorm(r, w, 0.1)[0]) + np.sum(dsum * r)
    assert math.isclose(difference(f, r, d), np.sum(dx * d), rel_tol=1e-7, abs_tol=1e-8)
    f = lambda w: np.sum(dy * layer.rmsnorm(r, w, 0.1)[0])
    assert math.isclose(difference(f, w, d[0]), np.sum(dw * d[0]), rel_tol=1e-7, abs_tol=1e-8)


def test_swiglu_closed_forms_and_extremes():
    assert layer.swiglu(0.0, 5.0) == 0.0
    assert math.isclose(layer.swiglu(math.log(3.0), 2.0), math.log(3.0) * 0.75 * 2, rel_tol=1e-15)
    assert layer.swiglu(800.0, 1.0) == 800.0 and abs(layer.swiglu(-800.0, 1.0)) < 1e-300
    g = rng().standard_normal(100) * 4
    # silu(g) - silu(-g) = g
    assert np.allclose(layer.swiglu(g, 1.0) - layer.swiglu(-g, 1.0), g)


def test_swiglu_backward_is_the_derivative():
    g = rng(3)
    gate, up, dh, d = (3 * g.standard_normal((4, 50)) for _ in range(4))
    dgate, dup = layer.swiglu_backward(dh, gate, up)
    f = lambda x: np.sum(dh * layer.swiglu(x, up))
    assert math.isclose(difference(f, gate, d), np.sum(dgate * d), rel_tol=1e-7)
    f = lambda x: np.sum(dh * layer.swiglu(gate, x))
    assert math.isclose(difference(f, up, d), np.sum(dup * d), rel_tol=1e-7)


def test_grad_norm_and_factor():
    grads = [np.array([3.0]), np.array([[0.0, 4.0], [12.0, 0.0]], np.float32)]
    assert layer.grad_norm(grads) == 13.0
    exact = sum(Fraction(float(x)) ** 2 for g in grads for x in g.ravel())
    assert exact == 169
    assert layer.clip_factor(13.0, 6.5) == 0.5 and layer.clip_factor(13.0, 13.0) == 1.0
    assert layer.clip_factor(13.0, 20.0) == 1.0


def test_code_errors_accepts_the_quantiser_and_rejects_mistakes():
    y = rng(5).standard_normal((6, 256)).astype(np.float32)
    q, s = quant.quantize_act(y)
    assert layer.code_errors(q, s, y, 0.0, 128, False) == (0, 0)
    # a computation 2^-20 off is within a reach of 2^-19, and not of 2^-24
    off = (y * np.float32(1 + 2.0 ** -20)).astype(np.float32)
    q2, s2 = quant.quantize_act(off)
    assert layer.code_errors(q2, s2, y, np.abs(y) * 2.0 ** -19, 128, False) == (0, 0)
    assert layer.code_errors(q2, s2, y, np.abs(y) * 2.0 ** -24, 128, False)[0] > 0
    wrong = q.copy()
    wrong[2, 17] ^= 1  # the neighbouring code
    assert layer.code_errors(wrong, s, y, np.abs(y) * 2.0 ** -19, 128, False)[1] == 1
    assert layer.code_errors(q, np.roll(s, 1, 0), y, np.abs(y) * 2.0 ** -19, 128, False)[0] > 0
    rounded = (y.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)  # codes of a bf16 result
    q3, _ = quant.quantize_act(rounded)
    assert layer.code_errors(q3, s, y, np.abs(y) * 2.0 ** -19, 128, False)[1] > 10
    # a group of zeros, and one too small for a float32 scale, count as zeros
    tiny = np.zeros((1, 128))
    tiny[0, 3] = 1e-40
    assert layer.code_errors(np.zeros((1, 128), np.uint8), np.ones((1, 1), np.float32), tiny, 0.0, 128,
                             False) == (0, 0)


def test_code_errors_power_of_two():
    from oracle import mx
    y = rng(6).standard_normal((4, 128)).astype(np.float32)
    for group in (32, 128):
        q, s = mx.quantize_mx_act(y, group)
        assert layer.code_errors(q, s, y, 0.0, group, True) == (0, 0)
        assert layer.code_errors(q, s + 1, y, 0.0, group, True)[0] > 0
