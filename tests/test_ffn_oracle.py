"""Pins of the float64 oracle of the gated feed-forward block's operators:
hand-worked values, invariants, and every gradient against differences."""
import math

import numpy as np
import pytest

from oracle import ffn_oracle as O


def _diff(f, x, h=1e-5):
    """Central differences of a scalar function of an array."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        g[i] = (f(x + e) - f(x - e)) / (2 * h)
    return g


def test_rms_norm_values():
    y = O.rms_norm_forward([[3.0, 4.0], [0.0, 0.0]], eps=0.5)
    np.testing.assert_allclose(y, [[3 / math.sqrt(13), 4 / math.sqrt(13)], [0, 0]])
    np.testing.assert_allclose(O.e4m3_scale([[-896.0, 1.0], [0.0, 0.0]]), [2.0, 1.0])


def test_rms_norm_gradient_against_differences():
    rng = np.random.default_rng(0)
    v, dy, dt = rng.standard_normal((3, 2, 3, 6))
    w = 1 + 0.3 * rng.standard_normal(6)
    f = lambda v, w: float(np.sum(dy * O.rms_norm_forward(v, w, 1e-2)) + np.sum(dt * v))
    dv, dw = O.rms_norm_backward(v, dy, w, 1e-2, dt)
    np.testing.assert_allclose(dv, _diff(lambda a: f(a, w), v), atol=1e-8)
    np.testing.assert_allclose(dw, _diff(lambda a: f(v, a), w), atol=1e-8)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation(act):
    g = np.linspace(-12, 12, 97)
    ref = g / (1 + np.exp(-g)) if act == "silu" else \
        0.5 * g * (1 + np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    np.testing.assert_allclose(O.activation(act, g), ref, atol=1e-14)
    np.testing.assert_allclose(O.activation_slope(act, g), (O.activation(act, g + 1e-5) - O.activation(act, g - 1e-5)) / 2e-5, atol=1e-8)
    # far out nothing overflows, and small values keep their digits
    assert np.all(np.isfinite(O.activation_slope(act, np.array([-300.0, 300.0]))))
    assert O.activation("silu", np.array([-100.0]))[0] == pytest.approx(-100 * math.exp(-100), rel=1e-12)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_ffn_gradient_against_differences(act):
    rng = np.random.default_rng(1)
    M, D, F = 3, 4, 5
    x, wg, wu = rng.standard_normal((M, D)), rng.standard_normal((F, D)), rng.standard_normal((F, D))
    bg, bu, dout = rng.standard_normal(F), rng.standard_normal(F), rng.standard_normal((M, F))
    f = lambda x, wg, wu, bg, bu: float(np.sum(dout * O.gated_ffn_forward(x, wg, wu, bg, bu, act)[0]))
    _, g, u = O.gated_ffn_forward(x, wg, wu, bg, bu, act)
    got = O.gated_ffn_backward(x, wg, wu, g, u, dout, act)
    args = [x, wg, wu, bg, bu]
    for i, d in enumerate(got):
        np.testing.assert_allclose(d, _diff(lambda v: f(*args[:i], v, *args[i + 1:]), args[i]), atol=1e-7)


def test_gated_ffn_scales_are_the_values_they_stand_for():
    rng = np.random.default_rng(2)
    x, wg, wu = rng.standard_normal((2, 3)), rng.standard_normal((4, 3)), rng.standard_normal((4, 3))
    xs, gs, us = rng.uniform(0.5, 2, 2), rng.uniform(0.5, 2, 4), rng.uniform(0.5, 2, 4)
    a = O.gated_ffn_forward(x, wg, wu, x_scale=xs, gate_scale=gs, up_scale=us)
    b = O.gated_ffn_forward(x * xs[:, None], wg * gs[:, None], wu * us[:, None])
    for p, q in zip(a, b):
        np.testing.assert_allclose(p, q)


def test_grad_norm():
    assert O.grad_norm([np.array([3.0]), np.array([[0.0, 4.0]]), np.zeros(0)]) == pytest.approx(5.0)
    assert O.grad_norm([np.full(4, 1e200)]) == pytest.approx(2e200)
    assert O.grad_norm([np.full(4, 1e-200)]) == pytest.approx(2e-200)
    assert O.grad_norm([]) == 0 and O.clip_factor(0.0, 0.0) == 1.0
    assert O.clip_factor(4.0, 1.0) == 0.25 and O.clip_factor(1.0, 4.0) == 1.0
    assert O.clip_factor(float("inf"), 1.0) == 1.0 and O.clip_factor(float("nan"), 1.0) == 1.0
