"""Float64 CPU oracle of the operators beside the model: rotation of q and k by
positions with several axes behind a per-head RMS norm, and group norm of
channels-last activations, each with its gradient.

Plain numpy written from the definitions (rotary shape and style:
SGLang-Diffusion "Support New Diffusion Models", "Verify the Port"); it shares
no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def rope_tables(pos, axes, theta):
    """cos, sin [..., R/2] of positions [..., n_axes]: axis a owns axes[a] / 2
    consecutive pairs, the j-th of them at frequency theta^(-2j / axes[a])."""
    pos = np.asarray(pos, np.float64)
    ang = [pos[..., a:a + 1] * theta ** (-2.0 * np.arange(w // 2) / max(w, 1)) for a, w in enumerate(axes)]
    ang = np.concatenate(ang, -1)
    return np.cos(ang), np.sin(ang)


def rope_pairs(R, style):
    """Channel indices (first, second) of every pair."""
    p = np.arange(R // 2)
    return (2 * p, 2 * p + 1) if style == "interleaved" else (p, p + R // 2)


def rope_turn(x, cos, sin, style):
    """x [B, N, H, d] turned; cos, sin broadcast to [B, N, 1, R/2]."""
    i, j = rope_pairs(2 * cos.shape[-1], style)
    y = np.array(x, np.float64)
    a, b = y[..., i].copy(), y[..., j].copy()
    y[..., i] = a * cos - b * sin
    y[..., j] = a * sin + b * cos
    return y


def _tables(pos, axes, theta):
    c, s = rope_tables(pos, axes, theta)
    if c.ndim == 2:
        c, s = c[None], s[None]
    return c[:, :, None], s[:, :, None]


def rope_forward(x, pos, axes, theta=1e4, style="interleaved", weight=None, eps=1e-6):
    x = np.asarray(x, np.float64)
    c, s = _tables(pos, axes, theta)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return rope_turn(x, c, s, style)


def rope_backward(dy, pos, axes, theta=1e4, style="interleaved", x=None, weight=None, eps=1e-6):
    """(dx, dweight or None)."""
    c, s = _tables(pos, axes, theta)
    g = rope_turn(dy, c, -s, style)
    if weight is None:
        return g, None
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xhat = x * r
    h = g * w
    return r * (h - xhat * np.mean(h * xhat, -1, keepdims=True)), np.sum(g * xhat, (0, 1, 2))


def group_norm_forward(x, groups, weight=None, bias=None, eps=1e-6, act="none"):
    """x [B, P, C] -> (y, mean [B, G], rstd [B, G])."""
    x = np.asarray(x, np.float64)
    B, P, C = x.shape
    v = x.reshape(B, P, groups, C // groups)
    mean = v.mean((1, 3))
    var = np.mean((v - mean[:, None, :, None]) ** 2, (1, 3))
    rstd = 1 / np.sqrt(var + eps)
    z = ((v - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(B, P, C)
    if weight is not None:
        z = z * np.asarray(weight, np.float64)
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    return (silu(z) if act == "silu" else z), mean, rstd


def silu(z):
    return z / (1 + np.exp(-z))


def group_norm_backward(x, dy, mean, rstd, groups, weight=None, bias=None, act="none"):
    """(dx, dweight, dbias) with the statistics of the forward pass."""
    x, dz = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    B, P, C = x.shape
    n = C // groups
    w = np.ones(C) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(C) if bias is None else np.asarray(bias, np.float64)
    r = np.repeat(np.asarray(rstd, np.float64), n, 1)[:, None]
    xhat = (x - np.repeat(np.asarray(mean, np.float64), n, 1)[:, None]) * r
    if act == "silu":
        z = xhat * w + b
        sg = 1 / (1 + np.exp(-z))
        dz = dz * sg * (1 + z * (1 - sg))
    g = dz * w

    def over_group(v):
        return np.repeat(v.reshape(B, P, groups, n).mean((1, 3)), n, 1)[:, None]

    return r * (g - over_group(g) - xhat * over_group(g * xhat)), (dz * xhat).sum((0, 1)), dz.sum((0, 1))
