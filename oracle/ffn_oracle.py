"""Float64 CPU oracle of the operators of a gated feed-forward block: RMS norm
with the residual's addition (into e4m3 too), gated feed-forward, and the norm
of many gradients with their clipping.

Plain numpy written from the definitions; it shares no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def f64(v):
    return None if v is None else np.asarray(v, np.float64)


def rms_norm_forward(v, weight=None, eps=1e-6):
    """Norm of v [..., C] (the sum as it is kept)."""
    v = f64(v)
    y = v / np.sqrt(np.mean(v * v, -1, keepdims=True) + eps)
    return y if weight is None else y * f64(weight)


def e4m3_scale(y):
    """Scale of each row of y [..., C]: max |y| / 448, 1 for zeros."""
    top = np.max(np.abs(f64(y)), -1)
    return np.where(top > 0, top / E4M3_MAX, 1.0)


def rms_norm_backward(v, dy, weight=None, eps=1e-6, dtotal=None):
    """(dv, dweight): the gradient of x, and of the residual too."""
    v, dy = f64(v), f64(dy)
    w = np.ones(v.shape[-1]) if weight is None else f64(weight)
    r = 1 / np.sqrt(np.mean(v * v, -1, keepdims=True) + eps)
    t, g = v * r, dy * w
    dv = r * (g - t * np.mean(g * t, -1, keepdims=True))
    if dtotal is not None:
        dv = dv + f64(dtotal)
    return dv, np.sum(dy * t, tuple(range(v.ndim - 1)))


_C = 2 * math.sqrt(2 / math.pi)


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1, e) / (1 + e), np.where(z >= 0, e, 1) / (1 + e)   # and 1 - sigmoid


def _argument(act, g):
    """z with act(g) = g sigmoid(z), and dz/dg."""
    if act == "silu":
        return g, np.ones_like(g)
    return _C * (g + 0.044715 * g ** 3), _C * (1 + 3 * 0.044715 * g ** 2)


def activation(act, g):
    g = f64(g)
    return g * _sigmoid(_argument(act, g)[0])[0]


def activation_slope(act, g):
    g = f64(g)
    z, dz = _argument(act, g)
    s, rest = _sigmoid(z)
    return s + g * s * rest * dz


def gated_ffn_forward(x, w_gate, w_up, bias_gate=None, bias_up=None, act="silu", x_scale=None, gate_scale=None,
                      up_scale=None):
    """(out, gate, up) of x [M, D] and weights [F, D]."""
    x = f64(x) if x_scale is None else f64(x) * f64(x_scale)[:, None]
    pre = []
    for w, s, b in ((w_gate, gate_scale, bias_gate), (w_up, up_scale, bias_up)):
        w = f64(w) if s is None else f64(w) * f64(s)[:, None]
        pre.append(x @ w.T + (0 if b is None else f64(b)))
    return activation(act, pre[0]) * pre[1], pre[0], pre[1]


def gated_ffn_slopes(gate, up, dout, act="silu"):
    """Gradients of gate and up."""
    gate, up, dout = f64(gate), f64(up), f64(dout)
    return dout * up * activation_slope(act, gate), dout * activation(act, gate)


def gated_ffn_backward(x, w_gate, w_up, gate, up, dout, act="silu"):
    """(dx, dw_gate, dw_up, dbias_gate, dbias_up)."""
    dg, du = gated_ffn_slopes(gate, up, dout, act)
    return dg @ f64(w_gate) + du @ f64(w_up), dg.T @ f64(x), du.T @ f64(x), dg.sum(0), du.sum(0)


def grad_norm(grads):
    """2-norm of all values of all arrays, without overflow."""
    flat = [np.abs(f64(g)).ravel() for g in grads]
    top = max((float(np.max(g)) for g in flat if g.size), default=0.0)
    if top == 0 or not np.isfinite(top):
        return top
    return top * math.sqrt(math.fsum(float(np.sum((g / top) ** 2)) for g in flat))


def clip_factor(norm, max_norm):
    return max_norm / norm if np.isfinite(norm) and norm > max_norm else 1.0
