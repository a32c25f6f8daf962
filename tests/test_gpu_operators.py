"""The rotation and group-norm operators on the GPU against their float64
oracle: types, head widths, layouts, positions, ragged and single sizes,
strides, offsets past 32 bits, non-finite values, in-place calls, gradients,
captured graphs, streams, and both operators around an attention layer.

Tolerances.  Arithmetic is fp32, each output rounded once to its type: at most
finfo(t).eps / 2 of the value.  Below that stands fp32 rounding, 2^-24 a step,
of sums whose terms have magnitude S: RSTEPS steps of the rotation (cos and
sin within 2 steps each, two products and a sum, the norm's row sum of at most
8 serial additions and 5 shuffles, its square root and three products: under
32), GSTEPS of the group norm (32 folded additions, at most 64 joined, 3 in
xhat, 2 in z, 8 in the sigmoid, 4 in its derivative: under 128).
"""
import math

import numpy as np
import pytest

from diffusion_transformer_denoising_gb300 import dit
from oracle import operators_oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ULP = 2.0 ** -24
RSTEPS, GSTEPS = 32, 128
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
STYLE = {"interleaved": dit.ROPE_INTERLEAVED, "split": dit.ROPE_SPLIT}
ACT = {"none": dit.ACT_NONE, "silu": dit.ACT_SILU}


def n64(t):
    return t.detach().cpu().double().numpy()


def half_step(t):
    return torch.finfo(t.dtype).eps / 2


def subnormal(t):
    return float(torch.finfo(t.dtype).smallest_normal) * torch.finfo(t.dtype).eps


def near(got, ref, scale, steps, name=""):
    """|got - ref| <= half a step of got's type at ref, and `steps` fp32 roundings at `scale`."""
    g = n64(got)
    assert np.array_equal(np.isnan(g), np.isnan(ref)), name
    tol = half_step(got) * np.abs(ref) + steps * ULP * np.asarray(scale) * (1 + half_step(got)) + subnormal(got)
    err = np.abs(g - ref)
    bad = err > tol
    assert not np.any(bad), f"{name}: error {np.nanmax(err):.3e}, {np.nanmax(err / tol):.2f} of the bound"


def randn(rng, shape, dtype, scale=1.0, shift=0.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale + shift).to(DT[dtype]).cuda()


def weights(rng, n):
    return torch.from_numpy(1 + 0.3 * rng.standard_normal(n)).float().cuda()


# ------------------------------------------------------------------ rotation
def views(rng, layout, B, N, H, d, dtype, fill=True):
    """A [B, N, H, d] view of the layout."""
    def new(*shape):
        return randn(rng, shape, dtype) if fill else torch.full(shape, float("nan"), dtype=DT[dtype], device="cuda")
    if layout == "heads":
        return new(B, H, N, d).transpose(1, 2)
    if layout == "packed":
        return new(B, N, 3, H, d)[:, :, 1]
    if layout == "odd":      # rows that start anywhere
        return new(B, N, H, d + 1)[..., 1:]
    return new(B, N, H, d)


def positions(rng, kind, B, N, n):
    if kind == "float":
        return torch.from_numpy(rng.uniform(-300, 300, (N, n))).float().cuda()
    if kind == "far":
        return torch.from_numpy(rng.integers(-2**31, 2**31, (B, N, n))).to(torch.int32).cuda()
    shape = (B, N, n) if kind == "batch" else (N, n)
    return torch.from_numpy(rng.integers(0, 200, shape)).to(torch.int32).cuda()


def row_scale(x, w, eps):
    """Magnitude of a pair's terms in the forward: the head's largest value after the norm."""
    if w is not None:
        x = np.abs(x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w)
    return np.max(np.abs(x), -1, keepdims=True, initial=0)


ROPE_CASES = [
    # dtype, B, N, Hq, Hk, d, axes, style, layout, positions
    ("bf16", 1, 1, 12, 12, 128, (44, 42, 42), "interleaved", "tokens", "grid"),
    ("bf16", 2, 333, 12, 12, 128, (44, 42, 42), "interleaved", "packed", "batch"),
    ("f16", 2, 67, 8, 2, 128, (0, 48, 48), "split", "heads", "grid"),
    ("f32", 1, 64, 4, 4, 32, (0, 16, 16), "interleaved", "tokens", "grid"),
    ("f32", 3, 41, 5, 1, 72, (24, 24, 24), "split", "tokens", "float"),
    ("bf16", 1, 50, 3, 3, 80, (16, 32, 32), "split", "tokens", "grid"),
    ("bf16", 2, 17, 2, 1, 96, (32, 0, 30), "interleaved", "odd", "batch"),
    ("f16", 1, 29, 7, 7, 256, (256,), "split", "heads", "grid"),
    ("f32", 2, 19, 3, 1, 256, (64, 64, 64, 62), "interleaved", "tokens", "float"),
    ("f32", 1, 23, 1, 0, 2, (2,), "split", "tokens", "grid"),
    ("bf16", 1, 9, 2, 0, 14, (4, 6), "split", "tokens", "grid"),
    ("bf16", 1, 300, 3, 1, 64, (0, 0), "interleaved", "tokens", "grid"),       # nothing turned
    ("bf16", 1, 40, 24, 40, 64, (16, 16, 16), "split", "tokens", "batch"),     # R/2 = 24, 16 channels behind
    ("f16", 1, 2100, 1, 1, 160, (56, 52, 52), "interleaved", "packed", "grid"),
    ("f32", 1, 77, 2, 2, 128, (64, 64), "split", "odd", "far"),
]


@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_rope_forward_and_backward(case, norm):
    dtype, B, N, Hq, Hk, d, axes, style, layout, kind = case
    rng = np.random.default_rng(N * 1000 + d)
    pos = positions(rng, kind, B, N, len(axes))
    eps = 1e-3
    kw = dict(axes=axes, theta=1e4, style=STYLE[style], eps=eps)
    t = {}
    for name, H in (("q", Hq), ("k", Hk)):
        if H:
            t[name] = dict(x=views(rng, layout, B, N, H, d, dtype), dy=views(rng, layout, B, N, H, d, dtype),
                           y=views(rng, layout, B, N, H, d, dtype, fill=False), dx=views(rng, "tokens", B, N, H, d, dtype, False),
                           w=weights(rng, d) if norm else None, dw=torch.full((d,), float("nan"), device="cuda") if norm else None)
    none = dict(x=None, dy=None, y=None, dx=None, w=None, dw=None)
    q, k = t["q"], t.get("k", none)
    dit.dit_rope_forward(pos, q["x"], q["y"], k["x"], k["y"], q_weight=q["w"], k_weight=k["w"], **kw)
    dit.dit_rope_backward(pos, q["dy"], q["dx"], k["dy"], k["dx"], q=q["x"], k=k["x"], q_weight=q["w"], k_weight=k["w"],
                          dq_weight=q["dw"], dk_weight=k["dw"], **kw)
    torch.cuda.synchronize()
    p = n64(pos)
    for name, v in t.items():
        x, dy = n64(v["x"]), n64(v["dy"])
        w = None if v["w"] is None else n64(v["w"])
        ref = O.rope_forward(x, p, axes, 1e4, style, w, eps)
        near(v["y"], ref, row_scale(x, w, eps), RSTEPS, f"{name} forward")
        dx, dw = O.rope_backward(dy, p, axes, 1e4, style, x, w, eps)
        g = np.max(np.abs(dy), -1, keepdims=True)
        if w is None:
            near(v["dx"], dx, g, RSTEPS, f"{name} gradient")
            continue
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
        xh = np.max(np.abs(x * r), -1, keepdims=True)
        # dx = r (h - xhat mean(h xhat)): each of its terms, and the mean's own d terms
        near(v["dx"], dx, r * g * np.max(np.abs(w)) * 1.5 * (1 + xh * np.mean(np.abs(x * r), -1, keepdims=True)), RSTEPS,
             f"{name} gradient")
        # a serial sum of at most rows / 4 terms, then 32 groups, 64 partials and 32 warps
        terms = np.sum(np.abs(dy).max(-1, keepdims=True) * np.abs(x * r) * 1.5, (0, 1, 2))
        near(v["dw"], dw, terms, RSTEPS + 64, f"{name} weight gradient")


def test_rope_in_place_and_shared_inputs():
    rng = np.random.default_rng(5)
    pos = positions(rng, "grid", 1, 90, 2)
    kw = dict(axes=(32, 32), style=dit.ROPE_SPLIT)
    q, w = views(rng, "packed", 2, 90, 3, 64, "bf16"), weights(rng, 64)
    out = torch.empty(2, 90, 3, 64, dtype=torch.bfloat16, device="cuda")
    dit.dit_rope_forward(pos, q, out, q_weight=w, **kw)
    dit.dit_rope_forward(pos, q, q, q_weight=w, **kw)
    assert torch.equal(q, out)
    # gradient over its own input gradient, and over x
    x, dy = views(rng, "tokens", 2, 90, 3, 64, "bf16"), views(rng, "tokens", 2, 90, 3, 64, "bf16")
    ref, dw, dw2 = torch.empty_like(x), torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    dit.dit_rope_backward(pos, dy, ref, q=x, q_weight=w, dq_weight=dw, **kw)
    a = dy.clone()
    dit.dit_rope_backward(pos, a, a, q=x, q_weight=w, dq_weight=dw2, **kw)
    assert torch.equal(a, ref) and torch.equal(dw, dw2)
    b = x.clone()
    dit.dit_rope_backward(pos, dy, b, q=b, q_weight=w, dq_weight=dw2, **kw)
    assert torch.equal(b, ref) and torch.equal(dw, dw2)
    # an input expanded over heads and batch: one row read by all
    row = randn(rng, (1, 90, 1, 64), "bf16")
    wide = row.expand(2, 90, 3, 64)
    dit.dit_rope_forward(pos, wide, out, **kw)
    ref2 = torch.empty_like(out)
    dit.dit_rope_forward(pos, wide.contiguous(), ref2, **kw)
    assert torch.equal(out, ref2)


def test_rope_norm_of_one_tensor_only_and_the_other_plain():
    rng = np.random.default_rng(6)
    pos, kw = positions(rng, "grid", 1, 33, 1), dict(axes=(32,), eps=1e-6)
    q, k, w = randn(rng, (1, 33, 4, 32), "f32"), randn(rng, (1, 33, 2, 32), "f32"), weights(rng, 32)
    qo, ko, q1, k1 = (torch.empty_like(v) for v in (q, k, q, k))
    dit.dit_rope_forward(pos, q, qo, k, ko, k_weight=w, **kw)
    dit.dit_rope_forward(pos, q, q1, **kw)
    dit.dit_rope_forward(pos, k, k1, q_weight=w, **kw)
    assert torch.equal(qo, q1) and torch.equal(ko, k1)
    dqo, dko = torch.randn_like(q), torch.randn_like(k)
    dw, dw1 = torch.empty(32, device="cuda"), torch.empty(32, device="cuda")
    dit.dit_rope_backward(pos, dqo, qo, dko, ko, k=k, k_weight=w, dk_weight=dw, **kw)
    dit.dit_rope_backward(pos, dqo, q1, **kw)
    dit.dit_rope_backward(pos, dko, k1, q=k, q_weight=w, dq_weight=dw1, **kw)
    assert torch.equal(qo, q1) and torch.equal(ko, k1) and torch.equal(dw, dw1)


def test_rope_far_and_tiny_float_positions():
    # the whole range of fp32: the angle is taken modulo a turn exactly
    vals = [0.0, -0.0, 1e-45, 1e-30, 2.0**-70, 0.125, 1.0, 3.7, -17.25, 12345.678, 1e6, -9e8, 2.0**40, 2.0**62]
    pos = torch.tensor(vals, dtype=torch.float32, device="cuda")[:, None]
    x = torch.ones(1, len(vals), 1, 4, device="cuda")
    y = torch.empty_like(x)
    dit.dit_rope_forward(pos, x, y, axes=(4,), theta=64.0)
    from fractions import Fraction
    ref = np.empty((len(vals), 4))
    inv_turn = Fraction(1) / (2 * Fraction(math.pi).limit_denominator(10**40))
    for i, v in enumerate(vals):
        p = Fraction(float(np.float32(v)))
        for j, f in enumerate((1, 8)):
            # the frequency in turns as a double holds it, then exact
            turns = p * Fraction(float(np.float64(1.0 / f) * 0.15915494309189533577))
            a = 2 * math.pi * float(turns - math.floor(turns))
            ref[i, 2 * j], ref[i, 2 * j + 1] = math.cos(a) - math.sin(a), math.sin(a) + math.cos(a)
    near(y[0, :, 0], ref, 2.0, RSTEPS)
    for v in (float("nan"), float("inf"), -float("inf")):
        pos[3] = v
        dit.dit_rope_forward(pos, x, y, axes=(4,), theta=64.0)
        assert torch.isnan(y[0, 3]).all() and torch.isfinite(y[0, 4]).all()


def test_rope_non_finite_values_stay_in_their_pair_or_head():
    pos = torch.arange(5, dtype=torch.int32, device="cuda")[:, None]
    for style, mate in ((dit.ROPE_INTERLEAVED, 5), (dit.ROPE_SPLIT, 12)):
        for bad in (float("nan"), float("inf")):
            x = torch.ones(1, 5, 2, 32, device="cuda")
            x[0, 2, 1, 4] = bad
            x[0, 3, 0, 30] = bad                  # behind the turned channels
            y = torch.empty_like(x)
            dit.dit_rope_forward(pos, x, y, axes=(16,), style=style)
            off = (~torch.isfinite(y)).nonzero().tolist()
            assert off == [[0, 2, 1, 4], [0, 2, 1, mate], [0, 3, 0, 30]], (style, off)
            dit.dit_rope_forward(pos, x, y, axes=(16,), style=style, q_weight=torch.ones(32, device="cuda"))
            rows = (~torch.isfinite(y)).any(-1).nonzero().tolist()
            assert rows == [[0, 2, 1], [0, 3, 0]], rows


def test_rope_zero_row_and_zero_tokens():
    pos = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    x, w = torch.zeros(1, 4, 1, 32, device="cuda"), torch.ones(32, device="cuda")
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.full((32,), 7.0, device="cuda")
    dit.dit_rope_forward(pos, x, y, axes=(32,), q_weight=w, eps=1e-6)
    assert (y == 0).all()
    dit.dit_rope_backward(pos, torch.ones_like(x), dx, axes=(32,), q=x, q_weight=w, dq_weight=dw, eps=1e-6)
    near(dx, np.full(x.shape, 1e3), 1e3, RSTEPS)
    assert (dw == 0).all()
    e = x[:, :0]
    dw.fill_(7.0)
    dit.dit_rope_forward(pos[:0], e, e, axes=(32,))
    dit.dit_rope_backward(pos[:0], e, e, axes=(32,), q=e, q_weight=w, dq_weight=dw)
    assert (dw == 0).all()


def test_rope_offsets_past_32_bits():
    buf = torch.empty(2**32 + 2**20, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(8)
    x = randn(rng, (2, 6, 2, 64), "bf16")
    pos = positions(rng, "grid", 2, 6, 2)
    far = buf.as_strided((2, 6, 2, 64), (2**32, 64, 2**16, 1))
    ref = torch.empty_like(x)
    kw = dict(axes=(32, 32), q_weight=weights(rng, 64))
    far.copy_(x)
    dit.dit_rope_forward(pos, x, ref, **kw)
    dit.dit_rope_forward(pos, far, far, **kw)
    assert torch.equal(far, ref)


# ------------------------------------------------------------------ group norm
GN_CASES = [
    # dtype, shape [B, ..., C], groups, act, affine, pad, shift
    ("bf16", (2, 16, 16, 512), 32, "silu", True, 0, 0.5),
    ("bf16", (5, 13, 17, 384), 32, "silu", True, 0, 0.5),
    ("f16", (1, 3, 11, 7, 192), 32, "silu", True, 8, 0.0),
    ("f32", (3, 37 * 53, 60), 12, "silu", True, 4, 1.0),
    ("f32", (2, 1, 64), 8, "none", True, 0, 0.0),
    ("bf16", (1, 1, 32), 2, "silu", False, 0, 0.0),
    ("f32", (2, 201, 7), 7, "none", False, 0, 0.0),
    ("bf16", (3, 515, 33), 3, "silu", True, 5, 0.0),
    ("f16", (2, 129, 10), 1, "silu", True, 0, 0.0),
    ("f32", (1, 9, 2300), 1, "silu", True, 0, 0.0),
    ("bf16", (1, 5, 4352), 34, "none", True, 0, 0.0),
    ("bf16", (1, 4099, 128), 32, "silu", True, 0, 3.0),
    ("bf16", (70, 3, 64), 4, "silu", True, 0, 0.0),
    ("f32", (1, 2, 3), 3, "none", True, 0, 0.0),
    ("f16", (1, 70001, 16), 4, "silu", True, 0, 0.0),
    ("bf16", (2, 40000, 48), 16, "silu", True, 0, 0.0),
    ("bf16", (1, 5000, 2304), 32, "silu", True, 0, 0.0),        # several slabs of whole groups
    ("bf16", (3, 2500, 96), 32, "silu", True, 5, 0.0),          # rows of any alignment, streamed
    ("f16", (2, 9001, 66), 6, "none", True, 0, 0.0),            # rows of 4-byte alignment, streamed
    ("f32", (1, 3001, 1100), 1, "silu", True, 0, 0.0),          # one group wider than a block
    ("f32", (9, 4000, 32), 32, "silu", True, 0, 0.0),
    ("bf16", (19, 40, 48), 4, "silu", True, 0, 0.0),            # small maps, their weight sums in a second launch
    ("f32", (3, 700, 16), 2, "silu", True, 0, 0.0),
    ("bf16", (8, 30, 64), 8, "silu", True, 0, 0.0),             # a cluster that holds the whole batch
    ("f16", (2, 97, 52), 4, "none", True, 0, 0.0),
]


def gn_tensors(rng, dtype, shape, pad, shift):
    C = shape[-1]
    x = randn(rng, (*shape[:-1], C + pad), dtype, 1.0, shift)[..., :C]
    x += torch.from_numpy(rng.standard_normal(C)).to(DT[dtype]).cuda()
    return x, randn(rng, shape, dtype)


def gn_check(x, dy, groups, act, w, b, y, mean, rstd, dx, dw, db, eps):
    """Everything against the oracle; magnitudes of the terms as the tolerances' scale."""
    B, C = x.shape[0], x.shape[-1]
    X, DY = n64(x).reshape(B, -1, C), n64(dy).reshape(B, -1, C)
    P, n = X.shape[1], C // groups
    W, Bi = (None if v is None else n64(v) for v in (w, b))
    ref, m, r = O.group_norm_forward(X, groups, W, Bi, eps, act)
    each = lambda v: np.repeat(v, n, 1)[:, None]
    dev = np.abs(X - each(m))
    dmax = dev.reshape(B, P, groups, n).max((1, 3))       # largest deviation of a group
    # mean: a sum of deviations; rstd: half the variance's relative error, the variance's terms up to dmax^2
    near(mean, m, np.abs(m) + dmax, GSTEPS, "mean")
    spread = (dmax * r) ** 2
    near(rstd, r, r * (1 + np.minimum(spread, P * n)), GSTEPS, "rstd")
    ww, bb = (np.ones(C) if W is None else np.abs(W)), (np.zeros(C) if Bi is None else np.abs(Bi))
    xs = each(dmax * r)
    zs = xs * ww + bb
    near(y, ref.reshape(n64(y).shape), (2 * zs).reshape(B, *[1] * (x.dim() - 2), C), GSTEPS, "y")
    # gradient from the statistics that the forward call wrote
    gx, gw, gb = O.group_norm_backward(X, DY, n64(mean), n64(rstd), groups, W, Bi, act)
    # |act'| <= 1.1 and |act''| <= 0.5: dz is off by steps of dy (1.1 + z / 2)
    dz = np.abs(DY) * (1.1 + zs / 2)
    g = (dz * ww).reshape(B, P, groups, n).max((1, 3))
    near(dx, gx.reshape(n64(dx).shape), (each(r * g) * (2 + xs * xs)).reshape(B, *[1] * (x.dim() - 2), C), GSTEPS, "dx")
    if dw is not None:
        # a serial part of at most 32 + P / 32 terms of one channel behind a join of 64
        near(dw, gw, (dz * xs).sum((0, 1)), GSTEPS, "dweight")
        near(db, gb, dz.sum((0, 1)), GSTEPS, "dbias")


@pytest.mark.parametrize("case", GN_CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_group_norm_forward_and_backward(case):
    dtype, shape, groups, act, affine, pad, shift = case
    rng = np.random.default_rng(shape[-1] * 10 + len(shape))
    x, dy = gn_tensors(rng, dtype, shape, pad, shift)
    C = shape[-1]
    w, b = (weights(rng, C), weights(rng, C) - 1) if affine else (None, None)
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")
    mean, rstd = nan(shape[0], groups), nan(shape[0], groups)
    dw, db = (nan(C), nan(C)) if affine else (None, None)
    y, dx = (torch.full(shape, float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
    dit.dit_group_norm_forward(x, y, groups, weight=w, bias=b, mean=mean, rstd=rstd, eps=1e-3, act=ACT[act])
    dit.dit_group_norm_backward(x, dy, mean, rstd, dx, groups, weight=w, bias=b, dweight=dw, dbias=db, act=ACT[act])
    torch.cuda.synchronize()
    gn_check(x, dy, groups, act, w, b, y, mean, rstd, dx, dw, db, 1e-3)
    # without statistics, and in place
    y2 = torch.empty_like(y)
    dit.dit_group_norm_forward(x, y2, groups, weight=w, bias=b, eps=1e-3, act=ACT[act])
    assert torch.equal(y, y2)
    dy2 = dy.clone()
    dit.dit_group_norm_backward(x, dy2, mean, rstd, dy2, groups, weight=w, bias=b, act=ACT[act])
    assert torch.equal(dy2, dx)
    inner = x.clone() if pad == 0 else x
    dit.dit_group_norm_forward(inner, inner, groups, weight=w, bias=b, eps=1e-3, act=ACT[act])
    assert torch.equal(inner, y)


def test_group_norm_large_mean_loses_nothing():
    # mean 1000 deviations away: sums of squares would lose every digit
    rng = np.random.default_rng(11)
    x = torch.from_numpy(1000 + rng.standard_normal((2, 3000, 32))).float().cuda()
    y, mean, rstd = torch.empty_like(x), torch.empty(2, 4, device="cuda"), torch.empty(2, 4, device="cuda")
    dit.dit_group_norm_forward(x, y, 4, mean=mean, rstd=rstd, eps=0.0)
    ref, m, r = O.group_norm_forward(n64(x), 4, eps=0.0)
    near(rstd, r, r * 25, GSTEPS)
    # xhat is off by the rounding of the mean itself, 1000 * 2^-24 deviations
    near(y, ref, 1000.0, 4)


def test_group_norm_mean_of_cancelling_channels():
    # channels near +-1 whose group mean is 1e-4: as good as the terms' own rounding allows, not as their size
    rng = np.random.default_rng(18)
    for P in (50, 20000):
        x = torch.from_numpy(np.where(np.arange(16) % 2, 1.0, -1.0) + 1e-3 * rng.standard_normal((3, P, 16)) + 1e-4).float().cuda()
        y, mean, rstd = torch.empty_like(x), torch.empty(3, 2, device="cuda"), torch.empty(3, 2, device="cuda")
        dit.dit_group_norm_forward(x, y, 2, mean=mean, rstd=rstd, eps=0.0)
        ref, m, r = O.group_norm_forward(n64(x), 2, eps=0.0)
        # deviations of 1e-3 summed in fp32, the result rounded once
        near(mean, m, np.abs(m) + 4e-3, 1)


def test_group_norm_non_finite_values_stay_in_their_group():
    for bad in (float("nan"), float("inf")):
        for P in (9, 5000):
            x = torch.randn(2, P, 32, device="cuda")
            x[1, P // 2, 9] = bad
            y, mean, rstd = torch.empty_like(x), torch.empty(2, 4, device="cuda"), torch.empty(2, 4, device="cuda")
            dit.dit_group_norm_forward(x, y, 4, mean=mean, rstd=rstd)
            off = torch.isnan(mean) if math.isnan(bad) else mean == bad
            assert off.nonzero().tolist() == [[1, 1]] and torch.isnan(rstd).nonzero().tolist() == [[1, 1]]
            hit = torch.isnan(y).all(1)
            assert hit[1, 8:16].all() and hit.sum() == 8, (bad, P)
            assert torch.isnan(y).sum() == 8 * P


def test_group_norm_constant_group_and_no_pixels():
    x = torch.full((1, 50, 8), 3.25, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(1, 2, device="cuda"), torch.empty(1, 2, device="cuda")
    dit.dit_group_norm_forward(x, y, 2, mean=mean, rstd=rstd, eps=1e-4)
    assert (y == 0).all() and (mean == 3.25).all()
    near(rstd, np.full((1, 2), 1 / math.sqrt(np.float32(1e-4))), 100.0, 8)
    e = x[:, :0]
    w, dw, db = torch.ones(8, device="cuda"), torch.full((8,), 7.0, device="cuda"), torch.full((8,), 7.0, device="cuda")
    dit.dit_group_norm_forward(e, e, 2, mean=mean, rstd=rstd, eps=1e-4)
    assert (mean == 0).all()
    dit.dit_group_norm_backward(e, e, mean, rstd, e, 2, weight=w, bias=w, dweight=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()
    dw.fill_(7.0)
    none, st = x[:0], mean[:0]
    dit.dit_group_norm_backward(none, none, st, st.clone(), none, 2, weight=w, bias=w, dweight=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()


def test_group_norm_offsets_past_32_bits():
    buf = torch.empty(2**32 + 2**22, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(12)
    x, dy = randn(rng, (2, 40, 64), "bf16"), randn(rng, (2, 40, 64), "bf16")
    far = buf.as_strided((2, 40, 64), (2**32, 2**16, 1))
    far.copy_(x)
    mean, rstd = torch.empty(2, 8, device="cuda"), torch.empty(2, 8, device="cuda")
    ref, dref, got, m2, r2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), mean.clone(), rstd.clone()
    dit.dit_group_norm_forward(x, ref, 8, mean=mean, rstd=rstd, act=dit.ACT_SILU)
    dit.dit_group_norm_backward(x, dy, mean, rstd, dref, 8, act=dit.ACT_SILU)
    dit.dit_group_norm_backward(far, dy, mean, rstd, got, 8, act=dit.ACT_SILU)
    assert torch.equal(got, dref)
    dit.dit_group_norm_forward(far, far, 8, mean=m2, rstd=r2, act=dit.ACT_SILU)
    assert torch.equal(far, ref) and torch.equal(m2, mean) and torch.equal(r2, rstd)


# ------------------------------------------------------------------ as a program uses them
def test_rows_around_a_view_are_left_alone():
    rng = np.random.default_rng(13)
    big = randn(rng, (4, 20, 3, 64), "bf16")
    before = big.clone()
    pos = positions(rng, "grid", 2, 12, 1)
    v = big[1:3, 4:16, 1:2]
    dit.dit_rope_forward(pos, v, v, axes=(64,))
    assert not torch.equal(big, before)
    big[1:3, 4:16, 1:2] = before[1:3, 4:16, 1:2]
    assert torch.equal(big, before)
    pix = randn(rng, (3, 50, 48), "bf16")
    before = pix.clone()
    v = pix[1:2, 10:40, 8:40]
    dit.dit_group_norm_forward(v, v, 4)
    pix[1:2, 10:40, 8:40] = before[1:2, 10:40, 8:40]
    assert torch.equal(pix, before)


@pytest.mark.parametrize("N,side", [(700, 60), (5000, 200), (40, 6)])  # every form of the kernels
def test_graph_replay_streams_and_repeated_calls_give_the_same_bits(N, side):
    rng = np.random.default_rng(14)
    pos = positions(rng, "grid", 1, N, 3)
    kw = dict(axes=(16, 24, 24), style=dit.ROPE_SPLIT)
    s = torch.cuda.Stream()

    def state(seed):
        g = np.random.default_rng(seed)
        x, dy = randn(g, (2, N, 4, 64), "bf16"), randn(g, (2, N, 4, 64), "bf16")
        f, df = randn(g, (2, side, 50, 96), "bf16"), randn(g, (2, side, 50, 96), "bf16")
        e = torch.empty
        return dict(x=x, dy=dy, w=weights(g, 64), y=torch.empty_like(x), dx=torch.empty_like(x), dw=e(64, device="cuda"),
                    f=f, df=df, fy=torch.empty_like(f), fdx=torch.empty_like(f), fw=weights(g, 96), fb=weights(g, 96),
                    fdw=e(96, device="cuda"), fdb=e(96, device="cuda"), m=e(2, 8, device="cuda"), r=e(2, 8, device="cuda"),
                    ws=e(max(dit.dit_group_norm_workspace_bytes(f, 8, True), dit.dit_group_norm_workspace_bytes(f, 8, False),
                             dit.dit_rope_workspace_bytes(64), 1), dtype=torch.uint8, device="cuda"))

    def go(t, stream=None):
        k = dict(workspace=t["ws"], stream=stream)
        dit.dit_rope_forward(pos, t["x"], t["y"], q_weight=t["w"], stream=stream, **kw)
        dit.dit_rope_backward(pos, t["dy"], t["dx"], q=t["x"], q_weight=t["w"], dq_weight=t["dw"], **k, **kw)
        dit.dit_group_norm_forward(t["f"], t["fy"], 8, weight=t["fw"], bias=t["fb"], mean=t["m"], rstd=t["r"],
                                   act=dit.ACT_SILU, **k)
        dit.dit_group_norm_backward(t["f"], t["df"], t["m"], t["r"], t["fdx"], 8, weight=t["fw"], bias=t["fb"],
                                    dweight=t["fdw"], dbias=t["fdb"], act=dit.ACT_SILU, **k)

    outs = ("y", "dx", "dw", "fy", "fdx", "fdw", "fdb", "m", "r")
    a, b = state(1), state(2)
    go(a)
    go(b)
    torch.cuda.synchronize()
    want_a, want_b = {k: a[k].clone() for k in outs}, {k: b[k].clone() for k in outs}
    for _ in range(3):                       # two streams at once, each with its own workspace
        for t in (a, b):
            for k in outs:
                t[k].zero_()
        s.wait_stream(torch.cuda.current_stream())
        go(a)
        go(b, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a[k], want_a[k]) and torch.equal(b[k], want_b[k]) for k in outs)
    g = torch.cuda.CUDAGraph()               # captured on one set of inputs, replayed on another
    with torch.cuda.graph(g):
        go(a)
    for k in ("x", "dy", "w", "f", "df", "fw", "fb"):
        a[k].copy_(b[k])
    for k in outs:
        a[k].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], want_b[k]) for k in outs)


def test_host_threads_call_at_once():
    # the same kernels with different shared memory, from four threads on a stream each
    import threading
    rng = np.random.default_rng(16)
    shapes = [(1, 64, 64, 64), (2, 32, 32, 256), (1, 40, 40, 512), (3, 150, 100, 64)]
    xs = [randn(rng, s, "bf16") for s in shapes]
    want = []
    for x in xs:
        y = torch.empty_like(x)
        dit.dit_group_norm_forward(x, y, 8, act=dit.ACT_SILU)
        want.append(y)
    ys = [torch.empty_like(x) for x in xs]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            ws = torch.empty(max(1, dit.dit_group_norm_workspace_bytes(xs[i], 8, False)), dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()
            for _ in range(50):
                dit.dit_group_norm_forward(xs[i], ys[i], 8, act=dit.ACT_SILU, workspace=ws, stream=s)
            s.synchronize()
        except Exception as e:  # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert all(torch.equal(a, b) for a, b in zip(ys, want))


def test_single_batch_element_of_an_odd_sized_batch():
    # the batch stride of one element says nothing about the rows' alignment
    rng = np.random.default_rng(17)
    x = randn(rng, (1, 33, 35, 64), "bf16")
    wide = torch.empty(2, 33 * 35 * 64 + 1, dtype=torch.bfloat16, device="cuda")[:1, :-1].view(1, 33, 35, 64)
    wide.copy_(x)
    y, z = torch.empty_like(x), torch.empty_like(x)
    dit.dit_group_norm_forward(x, y, 8)
    dit.dit_group_norm_forward(wide, z, 8)
    assert torch.equal(y, z)


def test_explicit_stream_needs_a_workspace():
    x = torch.randn(1, 100000, 32, device="cuda")
    s = torch.cuda.Stream()
    with pytest.raises(dit.DitError) as e:
        dit.dit_group_norm_backward(x, x, torch.zeros(1, 4, device="cuda"), torch.ones(1, 4, device="cuda"),
                                    torch.empty_like(x), 4, stream=s)
    assert e.value.status == dit.DIT_ERR_INVALID_ARG
    host = torch.zeros(4, 1, dtype=torch.int32).pin_memory()
    q = torch.zeros(1, 4, 1, 32, device="cuda")
    with pytest.raises(dit.DitError):
        dit.dit_rope_forward(host, q, q, axes=(32,))


def test_attention_block_of_a_latent_decoder():
    """Group norm + SiLU, projection, q/k norm + rotation over (h, w),
    attention, projection, residual: forward and every gradient, chained
    through both operators, against float64 autograd."""
    B, Hh, Ww, C, H, d, G = 2, 6, 5, 64, 2, 32, 8
    N = Hh * Ww
    rng = np.random.default_rng(15)
    new = lambda *s, k=1.0: torch.from_numpy(rng.standard_normal(s) * k).float().cuda()
    x, gw, gb, wqkv, wo = new(B, Hh, Ww, C), 1 + new(C, k=.2), new(C, k=.2), new(3 * C, C, k=.12), new(C, C, k=.12)
    qw, kw_ = 1 + new(d, k=.2), 1 + new(d, k=.2)
    dout = new(B, N, C)
    pos = torch.stack(torch.meshgrid(torch.arange(Hh), torch.arange(Ww), indexing="ij"), -1).reshape(N, 2).int().cuda()
    rope = dict(axes=(16, 16), theta=100.0, eps=1e-6)

    # the chain with the operators
    mean, rstd = torch.empty(2, B, G, device="cuda").unbind()
    h = torch.empty_like(x)
    dit.dit_group_norm_forward(x, h, G, weight=gw, bias=gb, mean=mean, rstd=rstd, eps=1e-5, act=dit.ACT_SILU)
    qkv = (h.reshape(B, N, C) @ wqkv.T).reshape(B, N, 3, H, d)
    q, k, v = qkv.unbind(2)
    qr, kr = torch.empty(2, B, N, H, d, device="cuda").unbind()
    dit.dit_rope_forward(pos, q, qr, k, kr, q_weight=qw, k_weight=kw_, **rope)
    s = torch.einsum("bnhd,bmhd->bhnm", qr, kr) / math.sqrt(d)
    p = s.softmax(-1)
    o = torch.einsum("bhnm,bmhd->bnhd", p, v).reshape(B, N, C)
    out = x.reshape(B, N, C) + o @ wo.T
    do = (dout @ wo).reshape(B, N, H, d)
    dp = torch.einsum("bnhd,bmhd->bhnm", do, v)
    ds = p * (dp - (dp * p).sum(-1, keepdim=True)) / math.sqrt(d)
    dqr, dkr = torch.einsum("bhnm,bmhd->bnhd", ds, kr), torch.einsum("bhnm,bnhd->bmhd", ds, qr)
    dqkv = torch.empty_like(qkv)
    dqw, dkw = torch.empty(2, d, device="cuda").unbind()
    dit.dit_rope_backward(pos, dqr.contiguous(), dqkv[:, :, 0], dkr.contiguous(), dqkv[:, :, 1], q=q, k=k, q_weight=qw,
                          k_weight=kw_, dq_weight=dqw, dk_weight=dkw, **rope)
    dqkv[:, :, 2] = torch.einsum("bhnm,bnhd->bmhd", p, do)
    flat = dqkv.reshape(B, N, 3 * C)
    dwqkv = torch.einsum("bno,bnc->oc", flat, h.reshape(B, N, C))
    dh = (flat @ wqkv).reshape(B, Hh, Ww, C)
    dx, dgw, dgb = torch.empty_like(x), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    dit.dit_group_norm_backward(x, dh, mean, rstd, dx, G, weight=gw, bias=gb, dweight=dgw, dbias=dgb, act=dit.ACT_SILU)
    dx += dout.reshape(B, Hh, Ww, C)

    # the same in float64, gradients by autograd
    X, GW, GB, WQ, WO, QW, KW = (t.cpu().double().requires_grad_() for t in (x, gw, gb, wqkv, wo, qw, kw_))
    V = X.reshape(B, N, G, C // G)
    var, mu = torch.var_mean(V, (1, 3), correction=0, keepdim=True)
    Z = ((V - mu) / (var + 1e-5).sqrt()).reshape(B, N, C) * GW + GB
    Q, K, VV = ((Z * Z.sigmoid()) @ WQ.T).reshape(B, N, 3, H, d).unbind(2)
    freq = torch.cat([100.0 ** (-torch.arange(0, 16, 2, dtype=torch.float64) / 16)] * 2)
    spin = torch.exp(1j * pos.cpu().double().repeat_interleave(8, 1) * freq)[None, :, None]

    def turn(t, w):
        t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        return torch.view_as_real(torch.view_as_complex(t.reshape(B, N, H, d // 2, 2)) * spin).flatten(-2)

    Qr, Kr = turn(Q, QW), turn(K, KW)
    Pm = (torch.einsum("bnhd,bmhd->bhnm", Qr, Kr) / math.sqrt(d)).softmax(-1)
    OUT = X.reshape(B, N, C) + torch.einsum("bhnm,bmhd->bnhd", Pm, VV).reshape(B, N, C) @ WO.T
    grads = torch.autograd.grad(OUT, (X, GW, GB, WQ, QW, KW), dout.cpu().double())
    pairs = [(out, OUT), *zip((dx, dgw, dgb, dwqkv, dqw, dkw), grads)]
    for i, (got, ref) in enumerate(pairs):
        ref = ref.detach().numpy()
        err = np.linalg.norm(n64(got) - ref) / np.linalg.norm(ref)
        # a chain of about a dozen fp32 stages, each a few steps of 2^-24 of its terms; sums over 60 rows and 64
        # channels may lose a factor of ten to cancellation
        assert err < 12 * 16 * 10 * ULP, (i, err)


def test_rope_in_place_at_the_most_rows():
    # 2^31 - 1 rows on 42 groups a block: every row is turned once
    N, d = 2**31 - 1, 48
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    if free < 2 * N * d + 2**33:
        pytest.skip(f"{free >> 30} GB free")
    pos = torch.ones(1, 1, dtype=torch.int32, device="cuda").expand(N, 1)
    row = torch.linspace(-2, 2, d, device="cuda").to(torch.bfloat16)
    want = torch.empty(1, 1, 1, d, dtype=torch.bfloat16, device="cuda")
    dit.dit_rope_forward(pos[:1], row.expand(1, 1, 1, d), want, axes=(d,))
    x = torch.empty(N, d, dtype=torch.bfloat16, device="cuda")
    x.copy_(row.expand(N, d))
    dit.dit_rope_forward(pos, x[None, :, None], x[None, :, None], axes=(d,))
    bad = [i for i in range(0, N, 2**24) if not (x[i:i + 2**24] == want[0, 0]).all()]
    del x
    torch.cuda.empty_cache()
    assert not bad, bad


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pixels", [2, 100, 60000], ids=["cluster", "cluster100", "streamed"])
def test_group_norm_silu_far_from_zero_on_its_own_scale(pixels, dtype):
    """xhat = +-1 exactly, so z = b +- w rounded once, and y = z sigma(z) to a count of steps of its own value: fp32
    16 (the exponential 4, the reciprocal 2, seven roundings, the sum 1 + e with e's own), its derivative s + z s (1 - s)
    (14 (1 + |z|) + 1) / |1 + z (1 - s)| < 20 for z < -8; 16 bits also 1.25 |z|, the rounding of the exponent."""
    C = 256
    z0 = np.linspace(-86, 40, C).astype(np.float32)
    x = torch.ones(1, pixels, C, dtype=DT[dtype], device="cuda")
    x[:, ::2] = -1
    w, b = torch.full((C,), 2.0**-12, device="cuda"), torch.from_numpy(z0).cuda()
    mean, rstd = torch.empty(1, 1, device="cuda"), torch.empty(1, 1, device="cuda")
    y = torch.empty_like(x)
    dit.dit_group_norm_forward(x, y, 1, weight=w, bias=b, mean=mean, rstd=rstd, eps=0.0, act=dit.ACT_SILU)
    assert mean.item() == 0 and rstd.item() == 1
    z = np.stack([(z0.astype(np.float64) - 2.0**-12), (z0.astype(np.float64) + 2.0**-12)]).astype(np.float32).astype(np.float64)
    s = 1 / (1 + np.exp(-z))
    steps = 16 + (0 if dtype == "f32" else 1.25) * np.abs(z)
    for p in (0, 1, pixels - 2, pixels - 1):
        near(y[0, p], (z * s)[p % 2], np.abs(z * s)[p % 2], steps[p % 2], f"y at pixel {p}")
    if pixels > 2:
        return
    dw, db, dx = torch.empty(C, device="cuda"), torch.empty(C, device="cuda"), torch.empty_like(x)
    dit.dit_group_norm_backward(x, torch.ones_like(x), mean, rstd, dx, 1, weight=w, bias=b, dweight=dw, dbias=db, act=dit.ACT_SILU)
    low = z0 < -8
    ref = (s * (1 + z * (1 - s))).sum(0)[low]
    near(db[torch.from_numpy(low).cuda()], ref, np.abs(ref), 24 + (0 if dtype == "f32" else 1.25 * np.abs(z0[low])), "dbias")


@pytest.mark.parametrize("style", ["interleaved", "split"])
@pytest.mark.parametrize("kind", ["int", "float"])
@pytest.mark.parametrize("theta", [1e4, 1e6])
def test_rope_sine_of_small_angles_on_its_own_scale(theta, kind, style):
    """Pairs (1, 0) turn to (cos, sin): each within 8 steps of 2^-24 of itself where it is not near 0, the sine of small
    angles too (the angle is rounded twice, then pi, a product, the polynomial's last sum)."""
    vals = [1, 2, -3, 17, 250] if kind == "int" else [0.015625, 0.7, 1.0, -2.3, 31.9]
    pos = torch.tensor(vals, dtype=torch.int32 if kind == "int" else torch.float32, device="cuda")[:, None]
    d = 128
    x = torch.zeros(1, len(vals), 2, d, device="cuda")
    i, j = O.rope_pairs(d, style)
    x[..., torch.from_numpy(i).cuda()] = 1
    y = torch.empty_like(x)
    dit.dit_rope_forward(pos, x, y, axes=(d,), theta=theta, style=STYLE[style])
    angle = n64(pos) * float(np.float32(theta)) ** (-2.0 * np.arange(d // 2) / d)
    ref = np.stack([np.cos(angle), np.sin(angle)], 0)[:, :, None].repeat(2, 2)
    got = np.stack([n64(y)[0][..., i], n64(y)[0][..., j]], 0)
    away = np.abs(ref) > np.abs(angle)[None, :, None] * 0.1     # off the zeros, where the angle's own steps count
    assert away.mean() > 0.8
    err = np.abs(got - ref) / np.abs(ref)
    assert err[away].max() < 8 * ULP, err[away].max() / ULP
    assert np.abs(got - ref).max() < 8 * ULP


PI = "3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803"


@pytest.mark.parametrize("kind", ["int", "float"])
@pytest.mark.parametrize("theta,axes", [(5.0, (256,)), (100.0, (256,)), (1e4, (256,)), (1.25, (64, 192)), (1e4, (44, 42, 42))])
def test_rope_far_positions_against_the_mathematical_angle(theta, axes, kind):
    """Angles in 80 decimal digits.  8 steps of 2^-24 in cos and sin, and the frequency's 2^-53 of an angle below 2^31
    (2^-22, 4 steps)."""
    from decimal import Decimal, getcontext
    getcontext().prec = 80
    vals = [2**31 - 1, -2**31, 2**30 + 12345, 987654321, -1234567] if kind == "int" else \
        [2.0**31, -9e8, 1.5e6 + 0.125, 123456.789, -2.0**30]
    pos = torch.tensor(vals, dtype=torch.int32 if kind == "int" else torch.float32, device="cuda")[:, None].repeat(1, len(axes))
    d = sum(axes)
    x = torch.zeros(1, len(vals), 1, d, device="cuda")
    x[..., ::2] = 1
    y = torch.empty_like(x)
    dit.dit_rope_forward(pos, x, y, axes=axes, theta=theta)
    turn, ref = 2 * Decimal(PI), np.empty((len(vals), d // 2, 2))
    freq = [Decimal(theta) ** (Decimal(-2 * j) / w) for w in axes for j in range(w // 2)]
    for i, v in enumerate(pos[:, 0].tolist()):
        for j, f in enumerate(freq):
            a = float((Decimal(v) * f) % turn)
            ref[i, j] = math.cos(a), math.sin(a)
    near(y[0, :, 0], ref.reshape(len(vals), d), 1.0, 12, "cos and sin")


@pytest.mark.parametrize("layout", ["tokens", "odd"])
def test_rope_weight_gradient_of_very_many_rows(layout):
    """One row 2.56 million times: equal terms, whose roundings do not cancel.  The bound is a sum of 33 rows, joined
    without loss, then 8 groups of a block, 10 partials a warp and 32 warps, and the term's own steps."""
    N, H, d = 40000, 64, 256
    rng = np.random.default_rng(21)
    x, dy = views(rng, layout, 1, 1, 1, d, "bf16"), views(rng, layout, 1, 1, 1, d, "bf16")
    pos, w = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), weights(rng, d)
    dx, dw = torch.empty(1, N, H, d, dtype=torch.bfloat16, device="cuda"), torch.empty(d, device="cuda")
    dit.dit_rope_backward(pos.expand(N, 1), dy.expand(1, N, H, d), dx, axes=(d,), q=x.expand(1, N, H, d), q_weight=w,
                          dq_weight=dw, eps=1e-6)
    _, ref = O.rope_backward(n64(dy), n64(pos), (d,), x=n64(x), weight=n64(w), eps=1e-6)
    near(dw, N * H * ref, N * H * np.abs(ref), 33 + 8 + 10 + 32 + RSTEPS, "weight gradient")
    # infinite terms stay where they are
    x = x.clone()
    dy = dy.clone()
    dy[..., 5] = float("inf")
    dit.dit_rope_backward(pos, dy, dx[:, :1, :1], axes=(d,), q=x, q_weight=w, dq_weight=dw, eps=1e-6)
    assert not torch.isfinite(dw[5]) and torch.isfinite(dw[6:]).all()


def streamed_cases():
    """Every run width of the three-launch form with enough pixels a thread that its loads ahead are refilled, unchecked
    batches run and remainders of 0, 1 and U - 1 pixels are left: q pixels for each thread of the writing pass, one more
    for some where `more`."""
    wide = [("bf16", 52, 13, 0, 4), ("f16", 60, 6, 0, 4), ("f32", 30, 5, 0, 2), ("bf16", 64, 8, 0, 8), ("f32", 32, 8, 0, 4)]
    short = [("f32", 27, 9, 0, 1), ("f32", 32, 8, 1, 1), ("bf16", 38, 2, 0, 2), ("f16", 48, 6, 2, 2), ("bf16", 31, 31, 0, 1),
             ("f16", 32, 4, 5, 1)]
    return [(*c, q, more) for c in wide for q, more in ((18, 1),)] + \
        [(*c, q, more) for c in short for q, more in ((16, 0), (17, 0), (23, 1))]


def form_check(monkeypatch, dtype, B, P, C, G, pad, forms):
    """Forward and gradient of one streamed case against the oracle, with the bound of the plans' own sums and 48 steps
    for xhat, z, the sigmoid, its derivative and the products."""
    from tests import group_norm_plan as plan
    rng = np.random.default_rng(C * 1000 + P)
    x, dy = gn_tensors(rng, dtype, (B, P, C), pad, 0.5)
    w, b = weights(rng, C), weights(rng, C) - 1
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")
    mean, rstd, dw, db = nan(B, G), nan(B, G), nan(C), nan(C)
    y, dx = (torch.full((B, P, C), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
    view = lambda t: (t.data_ptr(), t.stride(0) if B > 1 else 0, t.stride(1))
    e, steps = x.element_size(), 0
    for backward, out in ((False, y), (True, dx)):
        p = plan.plan(B, P, C, G, e, plan.vec_of(e, C, view(x), view(out), *([view(dy)] if backward else [])), backward)
        forms(p)
        steps = max(steps, plan.sum_steps(p, B, P, C, G, backward))
    monkeypatch.setitem(globals(), "GSTEPS", steps + 48)
    dit.dit_group_norm_forward(x, y, G, weight=w, bias=b, mean=mean, rstd=rstd, eps=1e-3, act=dit.ACT_SILU)
    dit.dit_group_norm_backward(x, dy, mean, rstd, dx, G, weight=w, bias=b, dweight=dw, dbias=db, act=dit.ACT_SILU)
    gn_check(x, dy, G, "silu", w, b, y, mean, rstd, dx, dw, db, 1e-3)


@pytest.mark.parametrize("case", streamed_cases(), ids=lambda c: "-".join(map(str, c)))
def test_group_norm_streams_of_every_run_width(case, monkeypatch):
    from tests import group_norm_plan as plan
    dtype, C, G, pad, vec, q, more = case
    e = 4 if dtype == "f32" else 2
    wave = plan.plan(1, 1 << 28, C, G, e, vec, False)
    step = wave["passes"] * wave["rows"]

    def forms(p):
        assert not p["cluster"] and p["vec"] == vec and p["passes"] * p["rows"] == step and p["pixels_a_thread"] == q + more

    form_check(monkeypatch, dtype, 1, step * q + more, C, G, pad, forms)


@pytest.mark.parametrize("case", [("f32", 170, 203, 1024, 32), ("bf16", 310, 260, 512, 16)], ids=lambda c: "-".join(map(str, c)))
def test_group_norm_long_sums_of_a_thread(case, monkeypatch):
    """More than one wave of work: what bounds a block's share is how many pixels a thread may sum in a row."""
    dtype, B, P, C, G = case

    def forms(p):
        assert not p["cluster"] and p["pixels_a_thread"] > (60 if dtype == "bf16" else 100)

    form_check(monkeypatch, dtype, B, P, C, G, 0, forms)


@pytest.mark.parametrize("B,P,C,G", [(200000, 1, 64, 4), (300, 700, 256, 2), (1, 1 << 24, 8, 1)], ids=["batch", "both", "pixels"])
def test_group_norm_weight_gradients_of_very_many_terms(B, P, C, G):
    """The same pixels in every batch element and equal gradients, so roundings do not cancel: a thread's sum of at most
    128 pixels and the rows of a block, then 128 splits and 128 batch elements and joins without loss (8 rows of a tree), and
    48 steps of the term itself."""
    rng = np.random.default_rng(22)
    one = rng.standard_normal((1, min(P, 700), C))
    x = torch.from_numpy(one).float().cuda()
    x = x.expand(B, *x.shape[1:]) if P <= 700 else x[:, :64].repeat(B, P // 64, 1)
    dy = torch.from_numpy(rng.uniform(1, 2, C)).float().cuda().expand(B, P, C)
    w, b = weights(rng, C), weights(rng, C) - 1
    mean, rstd, dx = torch.empty(B, G, device="cuda"), torch.empty(B, G, device="cuda"), torch.empty(B, P, C, device="cuda")
    dw, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    mean[:] = torch.from_numpy(rng.standard_normal(G)).float().cuda()
    rstd[:] = torch.from_numpy(rng.uniform(.5, 2, G)).float().cuda()
    dit.dit_group_norm_backward(x, dy, mean, rstd, dx, G, weight=w, bias=b, dweight=dw, dbias=db)
    xs = n64(x[:1, :min(P, 64 if P > 700 else 700)])
    _, gw, gb = O.group_norm_backward(xs, np.broadcast_to(n64(dy[0, 0]), xs.shape), n64(mean[:1]), n64(rstd[:1]), G, n64(w), n64(b))
    xhat = np.abs((xs - np.repeat(n64(mean[:1]), C // G, 1)[:, None]) * np.repeat(n64(rstd[:1]), C // G, 1)[:, None])
    times = B * P / xs.shape[1]
    near(db, times * gb, times * gb, 128 + 2 * 128 + 8 + 48, "dbias")
    near(dw, times * gw, times * (n64(dy[0, 0]) * xhat).sum((0, 1)), 128 + 2 * 128 + 8 + 48, "dweight")


def test_rope_gradient_of_q_and_k_in_different_layouts():
    """q by runs of 8 channels, k element by element (rows that start anywhere): two launches, k's partial weight sums
    behind q's; and both few enough for clusters."""
    rng = np.random.default_rng(23)
    for N, d, axes in ((1500, 128, (44, 42, 42)), (40, 128, (44, 42, 42)), (700, 64, (32, 32))):
        pos, kw = positions(rng, "grid", 2, N, len(axes)), dict(axes=axes, eps=1e-5)
        q, dyq = views(rng, "tokens", 2, N, 6, d, "bf16"), views(rng, "tokens", 2, N, 6, d, "bf16")
        k, dyk = views(rng, "odd", 2, N, 2, d, "bf16"), views(rng, "odd", 2, N, 2, d, "bf16")
        wq, wk = weights(rng, d), weights(rng, d)
        new = lambda: (torch.empty_like(q), torch.empty(2, N, 2, d, dtype=torch.bfloat16, device="cuda"),
                       torch.full((d,), float("nan"), device="cuda"), torch.full((d,), float("nan"), device="cuda"))
        dq, dk, dwq, dwk = new()
        dit.dit_rope_backward(pos, dyq, dq, dyk, dk, q=q, k=k, q_weight=wq, k_weight=wk, dq_weight=dwq, dk_weight=dwk, **kw)
        # each by itself gives the same rows; the sums are of other blocks
        eq, ek, ewq, ewk = new()
        dit.dit_rope_backward(pos, dyq, eq, q=q, q_weight=wq, dq_weight=ewq, **kw)
        dit.dit_rope_backward(pos, dyk, ek, q=k, q_weight=wk, dq_weight=ewk, **kw)
        assert torch.equal(dq, eq) and torch.equal(dk, ek)
        for x, dy, w, dw in ((q, dyq, wq, dwq), (k, dyk, wk, dwk)):
            _, ref = O.rope_backward(n64(dy), n64(pos), axes, x=n64(x), weight=n64(w), eps=1e-5)
            xh = np.abs(n64(x)) / np.sqrt(np.mean(n64(x) ** 2, -1, keepdims=True) + 1e-5)
            # 33 rows, 32 groups of a block, 19 partials a warp and 32 warps; the term's own steps
            near(dw, ref, np.sum(np.abs(n64(dy)).max(-1, keepdims=True) * xh * 1.5, (0, 1, 2)), 33 + 32 + 19 + 32 + RSTEPS)


def test_group_norm_of_the_most_pixels():
    """2^31 - 1 pixels of one channel: the counts of a thread and a block come close to 32 bits."""
    N = 2**31 - 1
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 8 * N + 2**33:
        pytest.skip("not enough memory free")
    x = torch.empty(1, N, 1, dtype=torch.bfloat16, device="cuda")
    x[0, :, 0] = 1.0
    x[0, ::2] = -1.0                                    # N odd: they cancel but for the last
    x[0, N - 1] = 3.0
    mean, rstd = torch.empty(1, 1, device="cuda"), torch.empty(1, 1, device="cuda")
    y = torch.empty_like(x)
    w, b = torch.full((1,), 2.0, device="cuda"), torch.full((1,), 0.5, device="cuda")
    dit.dit_group_norm_forward(x, y, 1, weight=w, bias=b, mean=mean, rstd=rstd, eps=0.0)
    assert abs(mean.item() - 3 / N) < 2**-12 and abs(rstd.item() - 1) < 2**-12
    want = torch.tensor([-1.5, 2.5], device="cuda").to(torch.bfloat16)
    pairs = y[0, :N - 1, 0].view(-1, 2)
    for i in range(0, len(pairs), 1 << 26):
        part = pairs[i:i + (1 << 26)]
        assert ((part.float() - want.float()).abs().amax() <= 2**-8 * 2.5), i
    assert abs(y[0, N - 1, 0].item() - 6.5) < 2**-8 * 6.5
    # gradient: dy = 1 everywhere, so dx is 0 but for what the sums leave, and dbias counts the pixels
    dy = torch.ones(1, 1, 1, dtype=torch.bfloat16, device="cuda").expand(1, N, 1)
    mean.zero_(), rstd.fill_(1.0)
    dw, db = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    dit.dit_group_norm_backward(x, dy, mean, rstd, y, 1, weight=w, bias=b, dweight=dw, dbias=db)
    assert db.item() == 2.0**31 and dw.item() == 3          # sums of +-1 that stay below 2^24 are exact
    assert y.abs().max() <= 2**-10
    del x, y, pairs, part
    torch.cuda.empty_cache()


def test_rope_weight_gradient_joined_without_loss():
    """One row in 128 groups of 304 blocks, at position 0 and with root 1, so a term is dy exactly: a lane adds two rows,
    eight groups are added as a tree (3), those joined without loss, a warp adds 10 partials, 32 warps a tree (5); two
    roundings of the results."""
    N, d = 2 * 128 * 304, 16
    rng = np.random.default_rng(24)
    dy = torch.from_numpy((1 + rng.integers(0, 2**23, (1, 1, 1, d)) * 2.0**-23)).float().cuda()
    x, w = torch.ones(1, 1, 1, d, device="cuda"), weights(rng, d)
    pos = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    dx, dw = torch.empty(1, N, 1, d, device="cuda"), torch.empty(d, device="cuda")
    dit.dit_rope_backward(pos.expand(N, 1), dy.expand(1, N, 1, d), dx, axes=(d,), q=x.expand(1, N, 1, d), q_weight=w,
                          dq_weight=dw, eps=0.0)
    ref = N * n64(dy)[0, 0, 0]
    near(dw, ref, ref, 2 + 3 + 10 + 5 + 2, "weight gradient")
