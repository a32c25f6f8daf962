"""Pins of the operators' float64 oracle: the rotation against complex numbers
and hand-worked angles, invariants, and every gradient against differences."""
import numpy as np
import pytest

from oracle import dit_oracle as D
from oracle import operators_oracle as O


def _diff(f, x, h=1e-5):
    """Central differences of a scalar function of an array."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        g[i] = (f(x + e) - f(x - e)) / (2 * h)
    return g


@pytest.mark.parametrize("style", ["interleaved", "split"])
def test_rotation_is_a_complex_product_per_pair(style):
    rng = np.random.default_rng(0)
    axes, d = (4, 0, 6), 14
    x = rng.standard_normal((2, 5, 3, d))
    pos = rng.integers(-50, 50, (2, 5, 3))
    y = O.rope_forward(x, pos, axes, 100.0, style)
    p = 0
    for a, w in enumerate(axes):
        for j in range(w // 2):
            i0, i1 = (2 * p, 2 * p + 1) if style == "interleaved" else (p, p + 5)
            spin = np.exp(1j * pos[..., a] * 100.0 ** (-2 * j / w))[:, :, None]
            z = (x[..., i0] + 1j * x[..., i1]) * spin
            np.testing.assert_allclose(y[..., i0], z.real, atol=1e-13)
            np.testing.assert_allclose(y[..., i1], z.imag, atol=1e-13)
            p += 1
    np.testing.assert_array_equal(y[..., 10:], x[..., 10:])


def test_rotation_agrees_with_the_model_oracle():
    # the same rotation as inside the model's blocks: interleaved, whole head, grid positions
    grid, axes = (2, 3, 4), (4, 6, 6)
    pos = np.stack(np.meshgrid(*[np.arange(n) for n in grid], indexing="ij"), -1).reshape(-1, 3)
    c, s = O.rope_tables(pos, axes, 1e4)
    x = np.random.default_rng(1).standard_normal((24, 16))
    ang = D.rope_angles(pos, axes, 1e4)
    np.testing.assert_allclose(c, np.cos(ang), atol=1e-14)
    np.testing.assert_allclose(s, np.sin(ang), atol=1e-14)
    y = O.rope_turn(x[None, :, None], c[None, :, None], s[None, :, None], "interleaved")
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x[None, :, None], axis=-1))


@pytest.mark.parametrize("style", ["interleaved", "split"])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_gradient_against_differences(style, norm):
    rng = np.random.default_rng(2)
    axes = (2, 4)
    x, dy = rng.standard_normal((2, 2, 2, 2, 8))
    pos = rng.integers(0, 30, (2, 2))
    w = 1 + 0.3 * rng.standard_normal(8) if norm else None
    f = lambda x, w: float(np.sum(dy * O.rope_forward(x, pos, axes, 50.0, style, w, 1e-3)))
    dx, dw = O.rope_backward(dy, pos, axes, 50.0, style, x, w, 1e-3)
    np.testing.assert_allclose(dx, _diff(lambda v: f(v, w), x), atol=1e-8)
    if norm:
        np.testing.assert_allclose(dw, _diff(lambda v: f(x, v), w), atol=1e-8)


@pytest.mark.parametrize("act", ["none", "silu"])
def test_group_norm_and_its_gradient(act):
    rng = np.random.default_rng(3)
    x = 2 + rng.standard_normal((2, 5, 6))
    dy = rng.standard_normal(x.shape)
    w, b = 1 + 0.3 * rng.standard_normal(6), rng.standard_normal(6)
    y, mean, rstd = O.group_norm_forward(x, 3, eps=0.0)
    v = y.reshape(2, 5, 3, 2)
    np.testing.assert_allclose(v.mean((1, 3)), 0, atol=1e-12)
    np.testing.assert_allclose(v.var((1, 3)), 1)
    f = lambda x, w, b: float(np.sum(dy * O.group_norm_forward(x, 3, w, b, 1e-2, act)[0]))
    _, mean, rstd = O.group_norm_forward(x, 3, eps=1e-2)
    dx, dw, db = O.group_norm_backward(x, dy, mean, rstd, 3, w, b, act)
    np.testing.assert_allclose(dx, _diff(lambda v: f(v, w, b), x), atol=1e-8)
    np.testing.assert_allclose(dw, _diff(lambda v: f(x, v, b), w), atol=1e-8)
    np.testing.assert_allclose(db, _diff(lambda v: f(x, w, v), b), atol=1e-8)
