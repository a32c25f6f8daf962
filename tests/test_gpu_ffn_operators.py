"""The operators of a gated feed-forward block on the GPU against their float64
oracle: types, widths, layouts, ragged and single sizes, strides, offsets past
32 bits, non-finite values, in-place calls, gradients, captured graphs, streams,
and all of them in the order a block uses them.

Tolerances.  Each output is rounded once to its type: at most finfo(t).eps / 2 of
the value, half a subnormal step below.  Below that stands fp32 rounding, 2^-24 a
step, of sums whose terms have magnitude S.
* RMS norm, NSTEPS: a row's sum of squares has at most 32 serial additions a
  thread, 5 shuffles and 32 joined warps, half of which counts in its square root,
  and five products: under 64.
* Products of D terms: at most 2 (D + 32) steps of the terms' absolute sum
  (truncating fp32 accumulation, one join).
* Activation, ASTEPS: the exponent z log2 e is rounded to 2^-24 of itself, at most
  2^-24 x 130 where the value is not zero, and doubled in z by GELU's cubic; two
  approximations of 2 steps each: under 512 steps of the value.
* The gradients of gate and up are rounded to the type as operands: half a step
  of each term more in dx and dw.
"""
import threading

import numpy as np
import pytest

from diffusion_transformer_denoising_gb300 import dit
from oracle import ffn_oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ULP = 2.0 ** -24
NSTEPS, ASTEPS = 64, 512
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
ACT = {"silu": dit.ACT_SILU, "gelu": dit.ACT_GELU}


def n64(t):
    return t.detach().float().cpu().double().numpy() if t.dtype is not torch.float32 else t.detach().cpu().double().numpy()


def half_step(t):
    return torch.finfo(t.dtype).eps / 2


def subnormal(t):
    return float(torch.finfo(t.dtype).smallest_normal) * torch.finfo(t.dtype).eps


def near(got, ref, err32, name=""):
    """|got - ref| <= half a step of got's type at ref, and err32 in front of that rounding."""
    g = n64(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.array_equal(np.isnan(g), np.isnan(ref)), name
    # past the type's largest number by more than its rounding and the error: infinite
    past = np.abs(ref) - err32 > torch.finfo(got.dtype).max * (1 + half_step(got))
    assert np.array_equal(g[past], np.sign(ref[past]) * np.inf), name
    g, ref = np.where(past, 0, g), np.where(past, 0, ref)
    tol = half_step(got) * np.abs(ref) + np.asarray(err32) * (1 + half_step(got)) + subnormal(got)
    err = np.abs(g - ref)
    bad = err > tol
    assert not np.any(bad), f"{name}: error {np.nanmax(err):.3e}, {np.nanmax(err / tol):.2f} of the bound at {np.argwhere(bad)[:3].tolist()}"


def randn(rng, shape, dtype, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(DT[dtype]).cuda()


def bits(t):
    return t.reshape(-1).view(torch.uint8)


def nans(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def padded(rng, shape, dtype, pad, fill=True):
    """A [..., C] slice of rows that are `pad` channels longer, starting at the pad's odd part."""
    wide = (*shape[:-1], shape[-1] + pad)
    t = randn(rng, wide, dtype) if fill else nans(wide, DT[dtype])
    off = pad % 2
    return t[..., off:off + shape[-1]]


# ------------------------------------------------------------------ rms norm
NORM_CASES = [
    # dtype, shape, residual, weight, pad
    ("bf16", (1, 1, 1536), True, True, 0), ("bf16", (2, 333, 1536), True, True, 0), ("f16", (3, 41, 512), False, True, 8),
    ("f32", (1, 7, 1), True, True, 0), ("bf16", (2, 5, 1), False, False, 0), ("f16", (1, 9, 7), True, True, 0),
    ("bf16", (1, 65, 8), True, True, 0), ("f32", (2, 33, 60), True, False, 0), ("bf16", (1, 50, 64), False, True, 1),
    ("f16", (2, 700, 255), True, True, 1), ("bf16", (1, 129, 256), True, True, 0), ("f32", (1, 300, 257), True, True, 3),
    ("f32", (3, 1237, 1001), False, True, 3), ("bf16", (1, 67, 1024), True, False, 0), ("bf16", (1, 67, 1026), True, True, 0),
    ("f16", (1, 31, 1535), True, True, 1), ("f32", (2, 19, 1536), True, True, 0), ("bf16", (2, 301, 2048), True, True, 0),
    ("bf16", (1, 29, 2056), True, True, 0), ("f32", (1, 29, 2050), True, True, 0), ("f16", (1, 23, 4096), True, True, 8),
    ("bf16", (1, 21, 5000), False, True, 1), ("f32", (1, 11, 8192), True, True, 0), ("bf16", (2, 5, 16384), True, True, 0),
    ("f32", (1, 5, 16384), True, True, 0), ("f16", (1, 5, 16383), True, False, 0), ("bf16", (5000, 1, 64), True, True, 0),
    ("bf16", (3, 77, 100), True, True, 1), ("f32", (2, 501, 13), True, True, 0), ("f16", (1, 999, 24), False, False, 1),
    ("bf16", (1, 9, 8200), True, True, 1), ("f32", (1, 13, 4099), True, True, 1), ("f16", (2, 11, 700), True, False, 3),
]


def norm_scale(v, w, eps):
    r = 1 / np.sqrt(np.mean(v * v, -1, keepdims=True) + eps)
    return r, np.abs(v * r) * (1 if w is None else np.abs(w))


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_rms_norm_forward_and_backward(case):
    dtype, shape, residual, affine, pad = case
    rng = np.random.default_rng(shape[-1] * 7 + shape[1])
    C, eps, t = shape[-1], 1e-3, DT[dtype]
    x, res = padded(rng, shape, dtype, pad), padded(rng, shape, dtype, pad) if residual else None
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(C)).float().cuda() if affine else None
    W = None if w is None else n64(w)
    total, out = padded(rng, shape, dtype, pad, fill=False) if residual else None, padded(rng, shape, dtype, pad, fill=False)
    dit.dit_rms_norm_forward(x, out, residual=res, total=total, weight=w, eps=eps)
    if residual:
        near(total, n64(x) + n64(res), ULP * (np.abs(n64(x)) + np.abs(n64(res))), "total")
    kept = total if residual else x
    v = n64(kept)
    ref = O.rms_norm_forward(v, W, eps)
    near(out, ref, NSTEPS * ULP * np.abs(ref), "out")
    # without the total, the norm is of the same sum
    out2 = torch.empty(shape, dtype=t, device="cuda")
    dit.dit_rms_norm_forward(x, out2, residual=res, weight=w, eps=eps)
    assert torch.equal(out2, out)
    # e4m3 with a scale for each row
    q, scale = torch.empty(shape, dtype=E4M3, device="cuda"), nans(shape[:-1], torch.float32)
    total8 = None if total is None else torch.empty(shape, dtype=t, device="cuda")
    dit.dit_rms_norm_forward(x, q, residual=res, total=total8, weight=w, scale=scale, eps=eps)
    if residual:
        assert torch.equal(total8, total)
    s = O.e4m3_scale(ref)
    near(scale, s, NSTEPS * ULP * s, "scale")
    near(q, ref / s[..., None], NSTEPS * ULP * np.abs(ref / s[..., None]), "e4m3")
    # gradient
    dy, dt = padded(rng, shape, dtype, pad), padded(rng, shape, dtype, pad) if residual else None
    dx, dw = padded(rng, shape, dtype, pad, fill=False), nans((C,), torch.float32) if affine else None
    dit.dit_rms_norm_backward(kept, dy, dx, dtotal=dt, weight=w, dweight=dw, eps=eps)
    DY = n64(dy)
    rdx, rdw = O.rms_norm_backward(v, DY, W, eps, None if dt is None else n64(dt))
    r, tn = norm_scale(v, None, eps)
    g = np.abs(DY * (1 if W is None else W))
    terms = r * (g + tn * np.mean(g * tn, -1, keepdims=True)) + (0 if dt is None else np.abs(n64(dt)))
    near(dx, rdx, NSTEPS * ULP * terms, "dx")
    if affine:
        # at most 256 rows one after the other, the rest without loss
        near(dw, rdw, (NSTEPS + 256) * ULP * np.sum(np.abs(DY) * tn, (0, 1)), "dweight")
    dx2 = torch.empty(shape, dtype=t, device="cuda")
    dit.dit_rms_norm_backward(kept, dy, dx2, dtotal=dt, weight=w, eps=eps)
    assert torch.equal(dx2, dx)


@pytest.mark.parametrize("C,pad", [(1536, 0), (77, 0), (77, 1), (2056, 0), (5000, 8)])
def test_rms_norm_in_place(C, pad):
    rng = np.random.default_rng(C)
    shape, w = (2, 37, C), torch.from_numpy(1 + 0.3 * rng.standard_normal(C)).float().cuda()
    x, res = padded(rng, shape, "bf16", pad), padded(rng, shape, "bf16", pad)
    total, out = torch.empty(shape, dtype=torch.bfloat16, device="cuda"), torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    dit.dit_rms_norm_forward(x, out, residual=res, total=total, weight=w)
    a, b = padded(rng, shape, "bf16", pad).copy_(x), padded(rng, shape, "bf16", pad).copy_(res)
    dit.dit_rms_norm_forward(a, a, residual=b, total=b, weight=w)
    assert torch.equal(a, out) and torch.equal(b, total)
    a.copy_(x), b.copy_(res)
    dit.dit_rms_norm_forward(a, b, residual=b, total=a, weight=w)
    assert torch.equal(b, out) and torch.equal(a, total)
    dy, dt = padded(rng, shape, "bf16", pad), padded(rng, shape, "bf16", pad)
    dx, dw, dw2 = torch.empty_like(out), nans((C,), torch.float32), nans((C,), torch.float32)
    dit.dit_rms_norm_backward(total, dy, dx, dtotal=dt, weight=w, dweight=dw)
    for k in range(3):
        v = [padded(rng, shape, "bf16", pad).copy_(t) for t in (total, dy, dt)]
        dit.dit_rms_norm_backward(v[0], v[1], v[k], dtotal=v[2], weight=w, dweight=dw2)
        assert torch.equal(v[k], dx) and torch.equal(dw, dw2), k


@pytest.mark.parametrize("dtype,C", [("bf16", 100), ("f16", 255), ("bf16", 768), ("f32", 1001), ("bf16", 1535), ("f16", 2056), ("bf16", 5000)])
@pytest.mark.parametrize("pads", [(0, 1, 3, 8), (1, 0, 8, 3), (8, 8, 1, 0)], ids=str)
def test_rms_norm_tensors_of_different_alignment(dtype, C, pads):
    rng = np.random.default_rng(C + pads[0])
    shape, w = (2, 19, C), torch.from_numpy(1 + 0.3 * rng.standard_normal(C)).float().cuda()
    x, res = padded(rng, shape, dtype, pads[0]), padded(rng, shape, dtype, pads[1])
    total, out = padded(rng, shape, dtype, pads[2], fill=False), padded(rng, shape, dtype, pads[3], fill=False)
    dit.dit_rms_norm_forward(x, out, residual=res, total=total, weight=w)
    near(total, n64(x) + n64(res), ULP * (np.abs(n64(x)) + np.abs(n64(res))), "total")
    ref = O.rms_norm_forward(n64(total), n64(w))
    near(out, ref, NSTEPS * ULP * np.abs(ref), "out")
    q, scale = torch.empty((2, 19, C + pads[0]), dtype=E4M3, device="cuda")[..., pads[0]:], nans((2, 19), torch.float32)
    total8 = padded(rng, shape, dtype, pads[3], fill=False)
    dit.dit_rms_norm_forward(x, q, residual=res, total=total8, weight=w, scale=scale)
    assert torch.equal(total8, total)
    s = O.e4m3_scale(ref)
    near(scale, s, NSTEPS * ULP * s, "scale")
    near(q, ref / s[..., None], NSTEPS * ULP * np.abs(ref / s[..., None]), "e4m3")
    dy, dx, dw = padded(rng, shape, dtype, pads[3]), padded(rng, shape, dtype, pads[1], fill=False), nans((C,), torch.float32)
    dit.dit_rms_norm_backward(total, dy, dx, dtotal=x, weight=w, dweight=dw)
    rdx, rdw = O.rms_norm_backward(n64(total), n64(dy), n64(w), 1e-6, n64(x))
    r, tn = norm_scale(n64(total), None, 1e-6)
    g = np.abs(n64(dy) * n64(w))
    near(dx, rdx, NSTEPS * ULP * (r * (g + tn * np.mean(g * tn, -1, keepdims=True)) + np.abs(n64(x))), "dx")
    near(dw, rdw, (NSTEPS + 38) * ULP * np.sum(np.abs(n64(dy)) * tn, (0, 1)), "dweight")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("C", [1, 2, 9, 33, 34, 60, 77, 130, 159])
@pytest.mark.parametrize("lefts", [(2, 2, 2, 2), (0, 2, 4, 6), (4, 0, 0, 2), (2, 2, 1, 2), (2, 3, 2, 2)], ids=str)
def test_rms_norm_rows_of_words(dtype, C, lefts):
    """Rows of an even stride that begin `left` channels into theirs: whole words, an odd last element, neighbours left alone."""
    rng = np.random.default_rng(C + 10 * sum(lefts))
    shape, w = (2, 35, C), torch.from_numpy(1 + 0.3 * rng.standard_normal(C)).float().cuda()
    width = (C + 7) // 2 * 2 + 2

    def rows(i, fill=True):
        wide = randn(rng, (*shape[:-1], width), dtype) if fill else torch.full((*shape[:-1], width), 7.0, dtype=DT[dtype], device="cuda")
        return wide, wide[..., lefts[i]:lefts[i] + C]

    def alone(wide, i):
        keep = wide.clone()
        keep[..., lefts[i]:lefts[i] + C] = 7.0
        assert torch.all(keep == 7.0)

    x, res = rows(0)[1], rows(1)[1]
    (wide_total, total), (wide_out, out) = rows(2, False), rows(3, False)
    dit.dit_rms_norm_forward(x, out, residual=res, total=total, weight=w)
    alone(wide_total, 2), alone(wide_out, 3)
    near(total, n64(x) + n64(res), ULP * (np.abs(n64(x)) + np.abs(n64(res))), "total")
    ref = O.rms_norm_forward(n64(total), n64(w))
    near(out, ref, NSTEPS * ULP * np.abs(ref), "out")
    q, scale = torch.empty(shape, dtype=E4M3, device="cuda"), nans((2, 35), torch.float32)
    dit.dit_rms_norm_forward(x, q, residual=res, weight=w, scale=scale)
    s = O.e4m3_scale(ref)
    near(scale, s, NSTEPS * ULP * s, "scale")
    near(q, ref / s[..., None], NSTEPS * ULP * np.abs(ref / s[..., None]), "e4m3")
    dy, (wide_dx, dx), dw = rows(3)[1], rows(1, False), nans((C,), torch.float32)
    dit.dit_rms_norm_backward(total, dy, dx, dtotal=x, weight=w, dweight=dw)
    alone(wide_dx, 1)
    rdx, rdw = O.rms_norm_backward(n64(total), n64(dy), n64(w), 1e-6, n64(x))
    r, tn = norm_scale(n64(total), None, 1e-6)
    g = np.abs(n64(dy) * n64(w))
    near(dx, rdx, NSTEPS * ULP * (r * (g + tn * np.mean(g * tn, -1, keepdims=True)) + np.abs(n64(x))), "dx")
    near(dw, rdw, (NSTEPS + 70) * ULP * np.sum(np.abs(n64(dy)) * tn, (0, 1)), "dweight")


@pytest.mark.parametrize("C", [30, 255, 1001, 2056, 5000])
def test_rms_norm_leaves_what_lies_around_its_rows_alone(C):
    rng = np.random.default_rng(C)
    for pad in (1, 3, 8):
        big = [torch.full((2, 9, C + pad + 16), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        view = [b[:, 1:-1, 5:5 + C] if pad != 8 else b[:, 1:-1, 8:8 + C] for b in big]
        x, res = randn(rng, (2, 7, C), "bf16"), randn(rng, (2, 7, C), "bf16")
        dit.dit_rms_norm_forward(x, view[0], residual=res, total=view[1])
        dit.dit_rms_norm_backward(x, res, view[2])
        for b, v in zip(big, view):
            assert not (v == 7).all()
            v.fill_(7.0)
            assert (b == 7).all()


def test_rms_norm_shared_inputs_and_shapes():
    # an input expanded over batch and tokens; one, two and four axes
    rng = np.random.default_rng(3)
    row = randn(rng, (1, 1, 96), "bf16")
    out = torch.empty(3, 5, 96, dtype=torch.bfloat16, device="cuda")
    one = torch.empty(96, dtype=torch.bfloat16, device="cuda")
    dit.dit_rms_norm_forward(row.expand(3, 5, 96), out)
    dit.dit_rms_norm_forward(row[0, 0], one)
    assert (out == one).all()
    x = randn(rng, (2, 3, 4, 96), "bf16")
    a, b = torch.empty_like(x), torch.empty_like(x)
    dit.dit_rms_norm_forward(x, a)
    dit.dit_rms_norm_forward(x.view(24, 96), b.view(24, 96))
    assert torch.equal(a, b)
    heads = x.transpose(0, 2)  # [4, 3, 2, 96]: no common stride behind the first axis
    with pytest.raises(dit.DitError):
        dit.dit_rms_norm_forward(heads, torch.empty_like(heads))


@pytest.mark.parametrize("C", [64, 77, 1536, 5000])
def test_rms_norm_rows_of_nan_infinity_and_zeros(C):
    rng = np.random.default_rng(C)
    x = randn(rng, (1, 9, C), "f32")
    x[0, 2, C // 2], x[0, 4, 0], x[0, 6] = float("nan"), float("inf"), 0.0
    w = torch.ones(C, device="cuda")
    good = [0, 1, 3, 5, 7, 8]
    out = nans(x.shape, torch.float32)
    dit.dit_rms_norm_forward(x, out, weight=w, eps=1e-6)
    assert torch.isnan(out[0, 2]).all() and torch.isnan(out[0, 4, 0]) and (out[0, 6] == 0).all()
    near(out[0, good], O.rms_norm_forward(n64(x[0, good])), 64 * ULP * np.abs(n64(out[0, good])))
    q, scale = torch.empty(x.shape, dtype=E4M3, device="cuda"), nans((1, 9), torch.float32)
    dit.dit_rms_norm_forward(x, q, weight=w, scale=scale, eps=1e-6)
    assert torch.isnan(scale[0, [2, 4]]).all() and (q[0, [2, 4]].float() == 0).all()
    assert scale[0, 6] == 1 and (q[0, 6].float() == 0).all()
    assert torch.isfinite(scale[0, good]).all() and (q[0, good].float().abs().amax(-1) == 448).all()
    dx, dw = nans(x.shape, torch.float32), nans((C,), torch.float32)
    dit.dit_rms_norm_backward(x, torch.ones_like(x), dx, weight=w, dweight=dw, eps=1e-6)
    assert torch.isnan(dx[0, 2]).all() and torch.isfinite(dx[0, good + [6]]).all()
    assert torch.isnan(dw[C // 2])


def test_rms_norm_e4m3_of_tiny_values():
    # scales stay normal numbers; values of 1e-44 have no digits left in them
    w = torch.full((32,), 1e-38, device="cuda")
    x = torch.ones(1, 3, 32, device="cuda")
    q, scale = torch.empty(1, 3, 32, dtype=E4M3, device="cuda"), nans((1, 3), torch.float32)
    dit.dit_rms_norm_forward(x, q, weight=w, scale=scale, eps=0.0)
    assert (scale == 2.0 ** -126).all()
    got = q.float().double() * scale.double()[..., None]
    assert ((got - 1e-38).abs() <= 1e-38 * 2.0 ** -4).all()


def test_rms_norm_without_rows():
    x, w, dw = torch.empty(2, 0, 16, device="cuda"), torch.ones(16, device="cuda"), torch.full((16,), 7.0, device="cuda")
    dit.dit_rms_norm_forward(x, x, weight=w)
    dit.dit_rms_norm_forward(x, x.to(E4M3), weight=w, scale=torch.empty(2, 0, device="cuda"))
    dit.dit_rms_norm_backward(x, x, x, weight=w, dweight=dw)
    assert (dw == 0).all()


@pytest.mark.parametrize("C", [64, 61, 2056])
def test_rms_norm_offsets_past_32_bits(C):
    buf = torch.empty(2**32 + 2**22, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(C)
    x, dy, w = randn(rng, (2, 6, C), "bf16"), randn(rng, (2, 6, C), "bf16"), torch.ones(C, device="cuda")
    far = buf.as_strided((2, 6, C), (2**32, 2**17, 1))
    ref, dx, dw, dw2 = torch.empty_like(x), torch.empty_like(x), nans((C,), torch.float32), nans((C,), torch.float32)
    dit.dit_rms_norm_forward(x, ref, weight=w)
    far.copy_(x)
    dit.dit_rms_norm_forward(far, far, weight=w)
    assert torch.equal(far, ref)
    dit.dit_rms_norm_backward(x, dy, dx, weight=w, dweight=dw)
    far.copy_(dy)
    dit.dit_rms_norm_backward(x, far, far, weight=w, dweight=dw2)
    assert torch.equal(far, dx) and torch.equal(dw, dw2)


def test_rms_norm_of_the_most_rows():
    n = 2**31 - 1
    row = torch.full((1, 1, 1), 3.0, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(1, n, 1, dtype=torch.bfloat16, device="cuda")
    dit.dit_rms_norm_forward(row.expand(1, n, 1), out, eps=0.0)
    assert out.min() == 1 and out.max() == 1
    with pytest.raises(dit.DitError):
        dit.dit_rms_norm_forward(row.expand(2, n, 1), out.expand(2, n, 1))


@pytest.mark.parametrize("rows,C", [(1 << 21, 8), (300_001, 77)])
def test_rms_norm_weight_gradient_of_very_many_rows(rows, C):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    x = torch.randn(rows, C, device="cuda", generator=g)
    dy = 1 + 0.01 * torch.randn(rows, C, device="cuda", generator=g)
    x.abs_()  # terms of one sign: a sum that grows
    dx, dw, w = torch.empty_like(x), nans((C,), torch.float32), torch.ones(C, device="cuda")
    dit.dit_rms_norm_backward(x, dy, dx, weight=w, dweight=dw)
    v = x.double()
    ref = (dy.double() * v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6)).sum(0).cpu().numpy()
    # 256 serial additions of terms of one sign round to at most half of that on the way
    near(dw, ref, (64 + 128) * ULP * ref, "dweight")


# ------------------------------------------------------------------ gated feed-forward
def matrix(rng, rows, cols, dtype, layout, scale=1.0):
    """plain; pitch: rows of 16-byte pitch in a wider buffer; odd: rows that start anywhere."""
    if layout == "plain":
        return randn(rng, (rows, cols), dtype, scale)
    pad = 8 - cols % 8 + 8 if layout == "pitch" else 3
    off = 0 if layout == "pitch" else 1
    return randn(rng, (rows, cols + pad), dtype, scale)[:, off:off + cols]


def quantised(t):
    s = torch.where(t.abs().amax(-1) > 0, t.abs().amax(-1).float() / 448, torch.ones((), device="cuda"))
    return (t.float() / s[:, None]).to(E4M3), s


FFN_CASES = [
    # dtype, rows, width, hidden, act, bias, layout
    ("bf16", 1, 1536, 520, "silu", False, "plain"), ("f16", 1, 7, 5, "silu", True, "odd"), ("bf16", 2, 1, 1, "gelu", True, "plain"),
    ("bf16", 8, 64, 16, "silu", False, "pitch"), ("f16", 9, 100, 17, "gelu", True, "odd"), ("bf16", 16, 65, 33, "silu", True, "plain"),
    ("f16", 17, 96, 40, "silu", False, "plain"), ("bf16", 32, 333, 129, "gelu", True, "plain"),
    ("bf16", 3, 64, 9760, "gelu", False, "plain"), ("f16", 30, 72, 9744, "silu", True, "plain"),   # more than one round of blocks
    ("bf16", 33, 64, 64, "silu", False, "plain"), ("f16", 33, 7, 5, "gelu", True, "odd"), ("bf16", 64, 1, 1, "silu", True, "plain"),
    ("bf16", 127, 65, 63, "silu", True, "pitch"), ("f16", 128, 64, 128, "gelu", False, "plain"), ("bf16", 129, 200, 130, "silu", True, "odd"),
    ("bf16", 255, 72, 264, "silu", False, "pitch"), ("f16", 257, 128, 257, "silu", True, "plain"), ("bf16", 300, 512, 520, "gelu", True, "plain"),
    ("bf16", 40, 4096, 64, "silu", True, "plain"),       # K split over CTAs
    ("f16", 70, 2050, 30, "gelu", False, "odd"),
    ("bf16", 2600, 256, 1280, "silu", False, "plain"),   # pairs of CTAs, several tiles each
    ("bf16", 1111, 136, 2100, "gelu", True, "plain"),
    ("bf16", 40, 64, 4096, "silu", True, "plain"),       # the gradients' K split: of dx,
    ("f16", 3000, 64, 72, "gelu", True, "plain"),        # and of dW
]


def forward_error(x, w, b, scales=(None, None)):
    """fp32 error of a projection, and the bound on its terms' absolute sum."""
    X = np.abs(n64(x)) * (1 if scales[0] is None else n64(scales[0])[:, None])
    W = np.abs(n64(w)) * (1 if scales[1] is None else n64(scales[1])[:, None])
    s = X @ W.T + (0 if b is None else np.abs(n64(b)))
    return 2 * (x.shape[1] + 32) * ULP * s


def check_forward(out, gate, up, x, wg, wu, bg, bu, act, xs=None, gs=None, us=None):
    ref, G, U = O.gated_ffn_forward(n64(x), n64(wg), n64(wu), None if bg is None else n64(bg), None if bu is None else n64(bu), act,
                                    *(None if s is None else n64(s) for s in (xs, gs, us)))
    eg, eu = forward_error(x, wg, bg, (xs, gs)), forward_error(x, wu, bu, (xs, us))
    a = np.abs(O.activation(act, G))
    # |act'| <= 1.13 for both activations
    near(out, ref, 1.13 * eg * (np.abs(U) + eu) + (a + 1.13 * eg) * eu + ASTEPS * ULP * a * np.abs(U), "out")
    if gate is not None:
        near(gate, G, eg, "gate")
        near(up, U, eu, "up")


@pytest.mark.parametrize("operands", ["same", "e4m3"])
@pytest.mark.parametrize("case", FFN_CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_gated_ffn_forward(case, operands):
    dtype, M, D, F, act, bias, layout = case
    rng = np.random.default_rng(M * 31 + D)
    x, both = matrix(rng, M, D, dtype, layout), matrix(rng, 2 * F, D, dtype, layout, 1.5 / D ** 0.5)
    kw = dict(act=ACT[act])
    scales = (None,) * 3
    if operands == "e4m3":
        (x, xs), (both, s) = quantised(x), quantised(both)
        if layout == "odd":
            x = torch.empty(M, D + 3, dtype=E4M3, device="cuda")[:, 1:1 + D].copy_(x)
        scales = xs, s[:F], s[F:]
        kw.update(x_scale=xs, gate_scale=s[:F], up_scale=s[F:])
    wg, wu = both[:F], both[F:]
    bg, bu = (torch.from_numpy(rng.standard_normal(F)).float().cuda() for _ in range(2)) if bias else (None, None)
    out, gate, up = (matrix(rng, M, F, dtype, layout).fill_(float("nan")) for _ in range(3))
    dit.dit_gated_ffn_forward(x, wg, wu, out, gate=gate, up=up, bias_gate=bg, bias_up=bu, **kw)
    check_forward(out, gate, up, x, wg, wu, bg, bu, act, *scales)
    out2 = nans((M, F), DT[dtype])
    dit.dit_gated_ffn_forward(x, wg, wu, out2, bias_gate=bg, bias_up=bu, **kw)
    assert torch.equal(out2, out)
    dit.dit_gated_ffn_synchronize()


@pytest.mark.parametrize("case", FFN_CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_gated_ffn_backward(case):
    dtype, M, D, F, act, bias, layout = case
    rng = np.random.default_rng(M * 17 + D)
    x, both = matrix(rng, M, D, dtype, layout), matrix(rng, 2 * F, D, dtype, layout, 1.5 / D ** 0.5)
    wg, wu = both[:F], both[F:]
    gate, up, dout = (matrix(rng, M, F, dtype, layout) for _ in range(3))
    dx, dwg, dwu = (matrix(rng, *s, dtype, layout).fill_(float("nan")) for s in ((M, D), (F, D), (F, D)))
    dbg, dbu = (nans((F,), torch.float32), nans((F,), torch.float32)) if bias else (None, None)
    args = (x, wg, wu, gate, up, dout)
    dit.dit_gated_ffn_backward(*args, dx=dx, dw_gate=dwg, dw_up=dwu, dbias_gate=dbg, dbias_up=dbu, act=ACT[act])
    ref = O.gated_ffn_backward(*(n64(t) for t in args), act)
    dg, du = O.gated_ffn_slopes(n64(gate), n64(up), n64(dout), act)
    h, X, Wg, Wu = half_step(x), np.abs(n64(x)), np.abs(n64(wg)), np.abs(n64(wu))
    # each slope: its approximation (|act'| and its terms are below 2.2), then half a step of the type
    eg = 2.2 * ASTEPS * ULP * np.abs(n64(dout) * n64(up))
    eu = ASTEPS * ULP * np.abs(du)
    tg, tu = (h * (np.abs(d) + e) + e + subnormal(x) for d, e in ((dg, eg), (du, eu)))
    near(dx, ref[0], tg @ Wg + tu @ Wu + 2 * (2 * F + 32) * ULP * (np.abs(dg) @ Wg + np.abs(du) @ Wu), "dx")
    near(dwg, ref[1], tg.T @ X + 2 * (M + 32) * ULP * np.abs(dg).T @ X, "dw_gate")
    near(dwu, ref[2], tu.T @ X + 2 * (M + 32) * ULP * np.abs(du).T @ X, "dw_up")
    if bias:
        # 32 rows one after the other and 8 joined, the blocks without loss
        near(dbg, ref[3], eg.sum(0) + 48 * ULP * np.abs(dg).sum(0), "dbias_gate")
        near(dbu, ref[4], eu.sum(0) + 48 * ULP * np.abs(du).sum(0), "dbias_up")
    # each output alone is the same
    for i, name in enumerate(("dx", "dw_gate", "dw_up", "dbias_gate", "dbias_up")):
        like = (dx, dwg, dwu, dbg, dbu)[i]
        if like is None:
            continue
        alone = nans(like.shape, like.dtype)
        dit.dit_gated_ffn_backward(*args, **{name: alone}, act=ACT[act])
        if name.startswith("dw"):
            # alone, a weight's gradient may split its rows over more CTAs: the same sums in another order
            near(alone, ref[i], (tg, tu)[i - 1].T @ X + 2 * (M + 32) * ULP * np.abs((dg, du)[i - 1]).T @ X, name)
        else:
            assert torch.equal(alone, like), name
    dit.dit_gated_ffn_synchronize()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [1, 200])
def test_gated_ffn_far_from_zero_on_its_own_scale(act, rows):
    # gate = x0, up = x1: the activation of every magnitude, small results with all their digits
    g = np.concatenate([np.linspace(-110, 110, 4001), -np.logspace(-6, 2, 400), np.array([1e4, 1e30, -1e4, -1e30, 0.0])])
    for dtype in ("bf16", "f16") if act == "silu" else ("bf16",):
        F = len(g)
        t = torch.from_numpy(np.clip(g, -6e4, 6e4) if dtype == "f16" else g).to(DT[dtype]).cuda()
        wg, wu = torch.stack([t, torch.zeros_like(t)], 1), torch.zeros(F, 2, dtype=DT[dtype], device="cuda")
        wu[:, 1] = 1
        x = torch.ones(rows, 2, dtype=DT[dtype], device="cuda")
        out = nans((rows, F), DT[dtype])
        dit.dit_gated_ffn_forward(x, wg, wu, out, act=ACT[act])
        ref = O.activation(act, n64(t))
        # GELU's z has three roundings more, cubed; and z of -90 is the last one above 2^-130
        near(out, np.broadcast_to(ref, (rows, F)), 2 * ASTEPS * ULP * np.abs(ref), f"{act} {dtype}")
        dg, du = nans((rows, F), DT[dtype]), nans((rows, F), DT[dtype])
        gate, one = t.expand(rows, F), torch.ones(rows, F, dtype=DT[dtype], device="cuda")
        db, du = nans((F,), torch.float32), nans((F,), torch.float32)
        dit.dit_gated_ffn_backward(x, wg, wu, gate, one, one, dbias_gate=db, dbias_up=du, act=ACT[act])
        slope = O.activation_slope(act, n64(t))
        z = np.minimum(np.abs(n64(t)), 1e4)
        s = np.abs(O.activation(act, n64(t)) / np.where(n64(t) == 0, 1, n64(t)))   # sigmoid
        terms = s * (1 + z * (1 if act == "silu" else 1.6 + 0.22 * z * z) * np.minimum(1, np.exp(-np.maximum(n64(t), 0)) * 2 + 0))
        near(db, rows * slope, rows * 4 * ASTEPS * ULP * terms + rows * 1e-36, f"{act} {dtype} slope")
        near(du, rows * ref, rows * 2 * ASTEPS * ULP * np.abs(ref) + rows * 2e-43, f"{act} {dtype} value")


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("operands", ["same", "e4m3"])
def test_gated_ffn_non_finite_values_stay_in_their_row_or_column(M, operands):
    rng = np.random.default_rng(M)
    D, F = 100, 150
    x, wg, wu = (randn(rng, s, "bf16", 0.3) for s in ((M, D), (F, D), (F, D)))
    kw = {}
    if operands == "e4m3":
        (x, xs), (wg, gs), (wu, us) = quantised(x), quantised(wg), quantised(wu)
        kw = dict(x_scale=xs, gate_scale=gs, up_scale=us)
    bad = float("nan")
    x[3, 7], wu[140, 99] = bad, bad
    out = torch.zeros(M, F, dtype=torch.bfloat16, device="cuda")
    dit.dit_gated_ffn_forward(x, wg, wu, out, **kw)
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[3], want[:, 140] = True, True
    assert torch.equal(nan, want)
    if operands == "e4m3":
        return
    x[3, 7], wu[140, 99] = 0, 0
    gate, up, dout = (randn(rng, (M, F), "bf16") for _ in range(3))
    gate[2, 149] = bad
    dx, dwg, dwu = (torch.zeros_like(t) for t in (x, wg, wu))
    db, du = torch.zeros(F, device="cuda"), torch.zeros(F, device="cuda")
    dit.dit_gated_ffn_backward(x, wg, wu, gate, up, dout, dx=dx, dw_gate=dwg, dw_up=dwu, dbias_gate=db, dbias_up=du)
    assert torch.isnan(dx).any(1).nonzero().flatten().tolist() == [2] and torch.isnan(dx[2]).all()
    for t in (dwg, dwu):
        assert torch.isnan(t).any(1).nonzero().flatten().tolist() == [149] and torch.isnan(t[149]).all()
    for t in (db, du):
        assert torch.isnan(t).nonzero().flatten().tolist() == [149]


def test_gated_ffn_without_rows():
    x, w = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda"), torch.ones(40, 24, dtype=torch.bfloat16, device="cuda")
    h = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    dit.dit_gated_ffn_forward(x, w, w.clone(), h)
    wide = torch.full((40, 30), 7.0, dtype=torch.bfloat16, device="cuda")
    dwg, dwu, db = wide[:, 3:27], torch.full_like(w, 7.0), torch.full((40,), 7.0, device="cuda")
    dit.dit_gated_ffn_backward(x, w, w.clone(), h, h, h, dx=x, dw_gate=dwg, dw_up=dwu, dbias_gate=db)
    assert (dwg == 0).all() and (dwu == 0).all() and (db == 0).all()
    assert (wide[:, :3] == 7).all() and (wide[:, 27:] == 7).all()


@pytest.mark.parametrize("M,D,F,layout", [(5, 64, 40, "plain"), (130, 72, 136, "pitch"), (130, 65, 67, "odd"), (40, 4096, 64, "pitch")])
def test_gated_ffn_leaves_what_lies_around_its_views_alone(M, D, F, layout):
    rng = np.random.default_rng(M)
    x, both = matrix(rng, M, D, "bf16", layout), matrix(rng, 2 * F, D, "bf16", layout, 0.1)
    gate, up, dout = (matrix(rng, M, F, "bf16", layout) for _ in range(3))
    def framed(rows, cols):
        big = torch.full((rows + 2, cols + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        return big, big[1:-1, 8 if layout != "odd" else 5:][:, :cols]
    def frame_kept(big, view):
        inner = torch.zeros_like(big, dtype=torch.bool)
        off = (view.data_ptr() - big.data_ptr()) // 2 - big.shape[1]
        inner[1:-1, off:off + view.shape[1]] = True
        return (big[~inner] == 7).all() and not (big[inner] == 7).all()
    outs = [framed(M, F) for _ in range(3)]
    dit.dit_gated_ffn_forward(x, both[:F], both[F:], outs[0][1], gate=outs[1][1], up=outs[2][1])
    grads = [framed(M, D), framed(F, D), framed(F, D)]
    dit.dit_gated_ffn_backward(x, both[:F], both[F:], gate, up, dout, dx=grads[0][1], dw_gate=grads[1][1], dw_up=grads[2][1])
    assert all(frame_kept(*v) for v in outs + grads)


def test_gated_ffn_shared_rows_and_more_axes():
    rng = np.random.default_rng(9)
    wg, wu = randn(rng, (72, 64), "bf16", 0.2), randn(rng, (72, 64), "bf16", 0.2)
    x = randn(rng, (1, 64), "bf16").expand(90, 64)       # one row for all
    out, ref = nans((90, 72), torch.bfloat16), nans((90, 72), torch.bfloat16)
    dit.dit_gated_ffn_forward(x, wg, wu, out)
    dit.dit_gated_ffn_forward(x.contiguous(), wg, wu, ref)
    assert torch.equal(out, ref)
    y = randn(rng, (3, 5, 6, 64), "bf16")
    o4, o2 = nans((3, 5, 6, 72), torch.bfloat16), nans((90, 72), torch.bfloat16)
    dit.dit_gated_ffn_forward(y, wg, wu, o4)
    dit.dit_gated_ffn_forward(y.view(90, 64), wg, wu, o2)
    assert torch.equal(o4.view(90, 72), o2)
    # the same weight twice, and dout that is gate and up as well
    dit.dit_gated_ffn_forward(y, wg, wg, o4)
    dwg, dwu = torch.empty_like(wg), torch.empty_like(wg)
    dit.dit_gated_ffn_backward(y, wg, wg, o4, o4, o4, dw_gate=dwg, dw_up=dwu)
    assert torch.isfinite(dwg.float()).all()


def test_gated_ffn_offsets_past_32_bits():
    buf = torch.empty(2**32 + 2**27, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(10)
    M, D, F = 65, 64, 72
    x, wg, wu = randn(rng, (M, D), "bf16"), randn(rng, (F, D), "bf16", 0.2), randn(rng, (F, D), "bf16", 0.2)
    ref = nans((M, F), torch.bfloat16)
    dit.dit_gated_ffn_forward(x, wg, wu, ref)
    for step in (2**26, 2**26 + 1):                      # tensor stores, plain stores; tensor loads, copies
        far = buf.as_strided((M, F), (step, 1))
        dit.dit_gated_ffn_forward(x, wg, wu, far)
        assert torch.equal(far, ref)
        fx = buf.as_strided((M, D), (step, 1))
        fx.copy_(x)
        out = nans((M, F), torch.bfloat16)
        dit.dit_gated_ffn_forward(fx, wg, wu, out)
        assert torch.equal(out, ref)
        few = nans((3, F), torch.bfloat16)
        dit.dit_gated_ffn_forward(fx[::32], wg, wu, few)  # rows 0, 32, 64 by the kernel of few rows
        assert (few.float() - ref[::32].float()).abs().max() <= 2.0 ** -7 * ref.float().abs().max()


def test_gated_ffn_gradients_of_more_than_4_gb_of_slopes():
    M, D, F = 140_000, 16, 8192                          # two slopes of 2.3 GB each
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    t = lambda *s: torch.randn(s, device="cuda", generator=g, dtype=torch.bfloat16)
    x, wg, wu, gate = t(M, D), t(F, D), t(F, D), t(M, F)
    one = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda").expand(M, F).contiguous()
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    db = nans((F,), torch.float32)
    dit.dit_gated_ffn_backward(x, wg, wu, gate, one, one, dx=dx, dw_gate=dwg, dw_up=dwu, dbias_up=db)
    last = slice(M - 50, M)
    dg, du = O.gated_ffn_slopes(n64(gate[last]), 1.0, 1.0)
    ref = dg @ n64(wg) + du @ n64(wu)
    terms = np.abs(dg) @ np.abs(n64(wg)) + np.abs(du) @ np.abs(n64(wu))
    near(dx[last], ref, (2.0 ** -9 + 2.0 ** -15 + 4 * F * ULP) * terms, "dx of the last rows")
    cols = [0, 5000, F - 1]
    dg, du = O.gated_ffn_slopes(n64(gate[:, cols]), 1.0, 1.0)
    # the last 64 columns of dw hold every row
    for got, d in ((dwg, dg), (dwu, du)):
        near(got[cols], d.T @ n64(x), (2.0 ** -9 + 2.0 ** -15 + 2 * M * ULP) * (np.abs(d).T @ np.abs(n64(x))), "dw")
    near(db[cols], du.sum(0), (2.0 ** -15 + 48 * ULP) * np.abs(du).sum(0), "dbias")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", [2e3, 2e2])
@pytest.mark.parametrize("rows", [70_001, 3_000_001, 20_000_003])
def test_gated_ffn_weight_gradient_of_very_many_rows(rows, size, dtype):
    # act(32) = 32 and 32 * dout are exact, and all terms of one sign: what is left is the sum of the products
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    D, F, t = 8, 8, DT[dtype]
    rand = lambda *s: torch.rand(s, device="cuda", generator=g)
    x, dout = (1 + rand(rows, D)).to(t), ((1 + rand(rows, F)) * (size / rows)).to(t)
    gate, up, w = torch.full((rows, F), 32.0, dtype=t, device="cuda"), torch.zeros(rows, F, dtype=t, device="cuda"), torch.zeros(F, D, dtype=t, device="cuda")
    dw, db = nans((F, D), t), nans((F,), torch.float32)
    dit.dit_gated_ffn_backward(x, w, w, gate, up, dout, dw_up=dw, dbias_up=db)
    ref, sums = np.zeros((F, D)), np.zeros(F)
    for i in range(0, rows, 1 << 22):
        d = dout[i:i + (1 << 22)].double() * 32
        ref += (d.t() @ x[i:i + (1 << 22)].double()).cpu().numpy()
        sums += d.sum(0).cpu().numpy()
    # 65536 rows are 4096 steps of the accumulator, each at most 2^-23 of the sum off, half of that on the way
    near(dw, ref, (2048 * 2 + 64) * ULP * ref, "dw")
    near(db, sums, 64 * ULP * sums, "dbias")


# ------------------------------------------------------------------ gradient norm
def grads(rng, shapes, scale=1.0):
    return [randn(rng, s, d, scale) for s, d in shapes]


GRAD_SETS = {
    "one": [((1,), "f32")],
    "few": [((3, 5), "bf16"), ((7,), "f32"), ((2049,), "f16"), ((64, 64), "bf16"), ((1, 1), "f16")],
    "empty": [((0,), "f32"), ((5,), "bf16"), ((3, 0), "bf16")],
    "large": [((1537, 4099), "bf16"), ((1_000_003,), "f32"), ((129, 70001), "f16")],
    "forty": [((97, 31), "bf16")] * 20 + [((33,), "f32")] * 20,
    "many": [((61,), "bf16")] * 900 + [((17000,), "f32")] * 500,
}


@pytest.mark.parametrize("name", GRAD_SETS)
def test_grad_norm_and_clipping(name):
    rng = np.random.default_rng(len(name))
    # parts of one buffer for each type: any alignment
    sizes = {d: sum(int(np.prod(s)) for s, t in GRAD_SETS[name] if t == d) for d in DT}
    flats, at, gs = {d: randn(rng, (n + 1,), d) for d, n in sizes.items()}, dict.fromkeys(DT, 1), []
    for s, d in GRAD_SETS[name]:
        n = int(np.prod(s))
        gs.append(flats[d][at[d]:at[d] + n].view(s))
        at[d] += n
    arrays = [n64(g) for g in gs]
    ref = O.grad_norm(arrays)
    norm = nans((), torch.float32)
    dit.dit_grad_norm(gs, norm)
    # 16 vectors of 8 squares in fp32, half of it in the root, the rest in fp64
    near(norm, np.array(ref), 72 * ULP * ref, "norm")
    outs = [nans(g.shape, g.dtype) for g in gs]
    for limit in (ref * 0.3, ref * 2, 0.0):
        again = nans((1,), torch.float32)
        dit.dit_grad_norm(gs, again, max_norm=limit, clipped=outs)
        assert again[0] == norm
        k = O.clip_factor(ref, limit)
        for o, a in zip(outs, arrays):
            near(o, a * k, 80 * ULP * np.abs(a * k), f"clipped {limit}")
    dit.dit_grad_norm(gs, norm, max_norm=ref * 2)         # below the limit: as they were
    for g, a in zip(gs, arrays):
        assert np.array_equal(n64(g), a)
    dit.dit_grad_norm(gs, again, max_norm=ref * 0.3, clipped=outs)
    dit.dit_grad_norm(gs, norm, max_norm=ref * 0.3)       # in place
    assert again[0] == norm and all(torch.equal(g, o) for g, o in zip(gs, outs))
    for d, f in flats.items():
        assert at[d] == sizes[d] + 1


@pytest.mark.parametrize("value,dtype", [(1e30, "f32"), (3e38, "f32"), (1e-30, "f32"), (1e-44, "f32"), (6e-8, "f16"), (65504.0, "f16"),
                                         (3e38, "bf16"), (1e-40, "bf16"), (1e15, "f32"), (1e-15, "f32")])
@pytest.mark.parametrize("n", [5, 4099])
def test_grad_norm_squares_neither_overflow_nor_vanish(value, dtype, n):
    g = torch.full((n,), value, dtype=DT[dtype], device="cuda")
    g[n // 2:] = 0
    norm = nans((), torch.float32)
    dit.dit_grad_norm([g], norm)
    ref = O.grad_norm([n64(g)])
    if ref > float(np.finfo(np.float32).max):
        assert torch.isinf(norm)
        return
    near(norm, np.array(ref), 72 * ULP * ref)
    out = torch.empty_like(g)
    dit.dit_grad_norm([g], norm, max_norm=ref / 2, clipped=[out])
    near(out, n64(g) * 0.5, 80 * ULP * n64(g) * 0.5 + 2.0 ** -149)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_grad_norm_that_is_not_finite_leaves_the_values(bad):
    g = torch.randn(5000, device="cuda")
    h = torch.randn(300, device="cuda").bfloat16()
    g[4321] = bad
    keep, keep_h, norm = g.clone(), h.clone(), torch.zeros((), device="cuda")
    dit.dit_grad_norm([g, h], norm, max_norm=1.0)
    assert (torch.isnan(norm) if bad != bad else torch.isinf(norm)) and torch.equal(g.view(torch.int32), keep.view(torch.int32)) and torch.equal(h, keep_h)
    out = [torch.zeros_like(g), torch.zeros_like(h)]
    dit.dit_grad_norm([g, h], norm, max_norm=1.0, clipped=out)
    assert torch.equal(out[0].nan_to_num(7.0), keep.nan_to_num(7.0)) and torch.equal(out[1], keep_h)


def test_grad_norm_of_nothing():
    norm = nans((), torch.float32)
    dit.dit_grad_norm([], norm)
    assert norm == 0
    norm.fill_(7)
    dit.dit_grad_norm([None, torch.empty(0, device="cuda")], norm, max_norm=1.0)
    assert norm == 0
    z = torch.zeros(10, device="cuda")
    dit.dit_grad_norm([z], norm, max_norm=0.0)
    assert norm == 0 and (z == 0).all()


def test_grad_norm_of_more_than_4_gb():
    g = torch.ones(2**31 + 12345, dtype=torch.bfloat16, device="cuda")
    norm = nans((), torch.float32)
    dit.dit_grad_norm([g], norm, max_norm=1024.0)
    ref = np.sqrt(2.0**31 + 12345)
    near(norm, np.array(ref), 72 * ULP * ref)
    want = torch.tensor(1024.0 / ref, dtype=torch.bfloat16)
    assert (g[:1000].cpu() == want).all() and g.min().cpu() == want and g.max().cpu() == want


# ------------------------------------------------------------------ together
def block_tensors(rng, M, D, F, dtype="bf16"):
    t = dict(x=randn(rng, (1, M, D), dtype), res=randn(rng, (1, M, D), dtype), w=torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).float().cuda(),
             wg=randn(rng, (F, D), dtype, 1 / D ** 0.5), wu=randn(rng, (F, D), dtype, 1 / D ** 0.5), dout=randn(rng, (1, M, F), dtype))
    like = lambda *s: torch.zeros(s, dtype=DT[dtype], device="cuda")
    t.update(total=like(1, M, D), y=like(1, M, D), h=like(1, M, F), gate=like(1, M, F), up=like(1, M, F), dy=like(1, M, D), dx=like(1, M, D),
             dwg=like(F, D), dwu=like(F, D), dw=torch.zeros(D, device="cuda"), norm=torch.zeros((), device="cuda"),
             q=torch.zeros(1, M, D, dtype=E4M3, device="cuda"), scale=torch.zeros(1, M, device="cuda"), h8=like(1, M, F))
    t["wg8"], t["gs"] = quantised(t["wg"])
    t["wu8"], t["us"] = quantised(t["wu"])
    return t


OUTPUTS = ("total", "y", "h", "gate", "up", "dy", "dx", "dwg", "dwu", "dw", "norm", "q", "scale", "h8")


def block_step(t, ws=None, stream=None):
    """A training step of the half block and a serving pass of it, as they follow each other."""
    kw = dict(stream=stream)
    ws = dict(kw, workspace=ws) if ws is not None else kw
    dit.dit_rms_norm_forward(t["x"], t["y"], residual=t["res"], total=t["total"], weight=t["w"], **kw)
    dit.dit_gated_ffn_forward(t["y"], t["wg"], t["wu"], t["h"], gate=t["gate"], up=t["up"], **ws)
    dit.dit_gated_ffn_backward(t["y"], t["wg"], t["wu"], t["gate"], t["up"], t["dout"], dx=t["dy"], dw_gate=t["dwg"], dw_up=t["dwu"], **ws)
    dit.dit_rms_norm_backward(t["total"], t["dy"], t["dx"], dtotal=t["x"], weight=t["w"], dweight=t["dw"], **ws)
    dit.dit_grad_norm([t["dwg"], t["dwu"], t["dw"]], t["norm"], max_norm=1.0, **ws)
    dit.dit_rms_norm_forward(t["x"], t["q"], residual=t["res"], weight=t["w"], scale=t["scale"], **kw)
    dit.dit_gated_ffn_forward(t["q"], t["wg8"], t["wu8"], t["h8"], x_scale=t["scale"], gate_scale=t["gs"], up_scale=t["us"], **ws)


@pytest.mark.parametrize("M,D,F,dtype", [(300, 256, 520, "bf16"), (1, 128, 96, "f16"), (77, 65, 131, "f16")])
def test_half_block_trained_and_served(M, D, F, dtype):
    rng = np.random.default_rng(M)
    t = block_tensors(rng, M, D, F, dtype)
    block_step(t)
    flat = {k: n64(v).reshape(-1, v.shape[-1]) if v.dim() == 3 else n64(v) for k, v in t.items()}
    h, ulp = half_step(t["x"]), ULP
    y = O.rms_norm_forward(flat["total"], flat["w"])
    near(t["y"][0], y, 64 * ulp * np.abs(y), "y")
    check_forward(t["h"][0], t["gate"][0], t["up"][0], t["y"][0], t["wg"], t["wu"], None, None, "silu")
    g = O.gated_ffn_backward(flat["y"], flat["wg"], flat["wu"], flat["gate"], flat["up"], flat["dout"])
    dg, du = (np.abs(v) for v in O.gated_ffn_slopes(flat["gate"], flat["up"], flat["dout"]))
    err = h + 2.0 ** -13 + 4 * (2 * F + M + 64) * ulp       # a slope's rounding, its approximation, the sums
    tiny = subnormal(t["x"])
    near(t["dy"][0], g[0], (err * dg + tiny + 2.0 ** -13 * np.abs(flat["dout"] * flat["up"])) @ np.abs(flat["wg"]) + (err * du + tiny) @ np.abs(flat["wu"]), "dy")
    dx, dw = O.rms_norm_backward(flat["total"], flat["dy"], flat["w"], dtotal=flat["x"])
    r, tn = norm_scale(flat["total"], None, 1e-6)
    dyw = np.abs(flat["dy"] * flat["w"])
    near(t["dx"][0], dx, 64 * ulp * (r * (dyw + tn * np.mean(dyw * tn, -1, keepdims=True)) + np.abs(flat["x"])), "dx")
    # the clipped gradients' own norm is the limit, but for their rounding
    clipped = O.grad_norm([flat["dwg"], flat["dwu"], flat["dw"]])
    assert n64(t["norm"]) > 1 and abs(clipped - 1) <= h + 200 * ulp + tiny * (2 * F * D + D) ** 0.5
    k = 1 / float(n64(t["norm"]))
    near(t["dw"], dw * k, (64 + 256 + 160) * ulp * np.sum(np.abs(flat["dy"]) * tn, 0) * k, "dw")
    check_forward(t["h8"][0], None, None, t["q"][0], t["wg8"], t["wu8"], None, None, "silu", t["scale"][0], t["gs"], t["us"])


@pytest.mark.parametrize("M,side", [(7, False), (300, False), (300, True)])
def test_graphs_streams_and_repeated_calls_give_the_same_bits(M, side):
    rng = np.random.default_rng(M)
    t, u = block_tensors(rng, M, 192, 264), block_tensors(rng, M + 5, 192, 264)
    block_step(t), block_step(u)
    torch.cuda.synchronize()
    ref = [{k: v[k].clone() for k in OUTPUTS} for v in (t, u)]
    ws = torch.empty(max(dit.dit_gated_ffn_workspace_bytes(v["y"], v["wg"], backward=True) for v in (t, u)) + (1 << 20),
                     dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    graphs = []
    for v in (t, u):                                       # two graphs that share a workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            block_step(v, ws)
        graphs.append(g)
    for _ in range(3):
        for v in (t, u):
            for k in OUTPUTS:
                v[k].zero_()
        ws.fill_(255)                                      # what it held means nothing
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for v, r in zip((t, u), ref):
            for k in OUTPUTS:
                assert torch.equal(bits(v[k]), bits(r[k])), k
    # eagerly on another stream, with the workspace passed in
    if side:
        for k in OUTPUTS:
            t[k].zero_()
        torch.cuda.synchronize()
        block_step(t, ws, stream=stream)
        torch.cuda.synchronize()
        for k in OUTPUTS:
            assert torch.equal(bits(t[k]), bits(ref[0][k])), k
    dit.dit_gated_ffn_synchronize()


def test_first_calls_of_a_process_inside_a_capture():
    """No call needs one outside of a capture before it."""
    code = """
import torch
from diffusion_transformer_denoising_gb300 import dit
def go(out):
    M, D, F = 300, 512, 768
    r = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda") * 0.125
    x, wg, wu, dout = r(1, M, D), r(F, D), r(F, D), r(1, M, F)
    e = torch.empty_like
    total, y, h, gate, up, dy, dx, dwg, dwu = e(x), e(x), e(dout), e(dout), e(dout), e(x), e(x), e(wg), e(wu)
    w, dw, norm = torch.ones(D, device="cuda"), torch.empty(D, device="cuda"), torch.empty((), device="cuda")
    def step():
        dit.dit_rms_norm_forward(x, y, residual=x, total=total, weight=w)
        dit.dit_gated_ffn_forward(y, wg, wu, h, gate=gate, up=up)
        dit.dit_gated_ffn_backward(y, wg, wu, gate, up, dout, dx=dy, dw_gate=dwg, dw_up=dwu)
        dit.dit_rms_norm_backward(total, dy, dx, weight=w, dweight=dw)
        dit.dit_grad_norm([dwg, dwu, dw], norm, max_norm=0.5)
    torch.cuda.synchronize()
    if out:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        g.replay()
    else:
        step()
    torch.cuda.synchronize()
    return [v.double().sum().item() for v in (h, dx, dwg, dwu, dw, norm)]
a = go(True)
assert a == go(False), a
print("same")
"""
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_host_threads_call_at_once():
    rng = np.random.default_rng(5)
    sets = [block_tensors(rng, m, 136, 200) for m in (3, 33, 150, 290)]
    for t in sets:
        block_step(t)
    torch.cuda.synchronize()
    ref = [{k: t[k].clone() for k in OUTPUTS} for t in sets]
    errors = []

    def work(t):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    block_step(t)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(t,)) for t in sets]
    [th.start() for th in threads]
    [th.join() for th in threads]
    torch.cuda.synchronize()
    assert not errors, errors
    for t, r in zip(sets, ref):
        for k in OUTPUTS:
            assert torch.equal(bits(t[k]), bits(r[k])), k


def test_explicit_stream_needs_a_workspace():
    rng = np.random.default_rng(6)
    t = block_tensors(rng, 40, 64, 72)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dit.dit_rms_norm_forward(t["x"], t["y"], residual=t["res"], total=t["total"], stream=s)      # needs none
    for call in (lambda **k: dit.dit_gated_ffn_backward(t["y"], t["wg"], t["wu"], t["gate"], t["up"], t["dout"], dx=t["dy"], **k),
                 lambda **k: dit.dit_rms_norm_backward(t["total"], t["dy"], t["dx"], weight=t["w"], dweight=t["dw"], **k),
                 lambda **k: dit.dit_grad_norm([t["dwg"]], t["norm"], **k)):
        with pytest.raises(dit.DitError):
            call(stream=s)
        call(stream=s, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    s.synchronize()
    with pytest.raises(dit.DitError):                      # host memory
        dit._check(dit.lib().dit_rms_norm_forward(dit._norm_args(t["x"].cpu(), None, None, None, t["y"].cpu(), torch.bfloat16, None, None, None, 1e-6), None))


def test_gradients_through_autograd_functions():
    """The calls inside a torch.autograd.Function, as a training program has them: directional differences of the
    whole half block against its gradient."""
    class HalfBlock(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, res, w, wg, wu):
            M, F = x.shape[1], wg.shape[0]
            total, y = torch.empty_like(x), torch.empty_like(x)
            h, gate, up = (torch.empty(1, M, F, dtype=x.dtype, device="cuda") for _ in range(3))
            dit.dit_rms_norm_forward(x, y, residual=res, total=total, weight=w)
            dit.dit_gated_ffn_forward(y, wg, wu, h, gate=gate, up=up)
            ctx.save_for_backward(total, y, w, wg, wu, gate, up)
            return total, h

        @staticmethod
        def backward(ctx, dtotal, dh):
            total, y, w, wg, wu, gate, up = ctx.saved_tensors
            dy, dx, dwg, dwu, dw = (torch.empty_like(t) for t in (y, y, wg, wu, w))
            dit.dit_gated_ffn_backward(y, wg, wu, gate, up, dh.contiguous(), dx=dy, dw_gate=dwg, dw_up=dwu)
            dit.dit_rms_norm_backward(total, dy, dx, dtotal=dtotal.contiguous(), weight=w, dweight=dw)
            return dx, dx, dw, dwg, dwu

    rng = np.random.default_rng(7)
    M, D, F = 33, 48, 80
    leaves = [randn(rng, (1, M, D), "f16"), randn(rng, (1, M, D), "f16"), torch.ones(D, device="cuda"),
              randn(rng, (F, D), "f16", 0.2), randn(rng, (F, D), "f16", 0.2)]
    for v in leaves:
        v.requires_grad_()
    dtotal, dh = randn(rng, (1, M, D), "f16"), randn(rng, (1, M, F), "f16")
    got = torch.autograd.grad(HalfBlock.apply(*leaves), leaves, (dtotal, dh))
    with pytest.raises(dit.DitError):                      # outside of it, autograd would not see the call
        dit.dit_gated_ffn_forward(leaves[0], leaves[3], leaves[4], torch.empty(1, M, F, dtype=torch.float16, device="cuda"))

    def loss(*v):
        total = v[0] + v[1]
        return np.sum(n64(dtotal)[0] * total) + np.sum(n64(dh)[0] * O.gated_ffn_forward(O.rms_norm_forward(total, v[2]), v[3], v[4])[0])

    at = [n64(v).reshape(-1, v.shape[-1]) if v.dim() > 1 else n64(v) for v in leaves]
    for i, (g, v) in enumerate(zip(got, at)):
        d = rng.standard_normal(v.shape)
        shift = lambda s: [a + s * 1e-5 * d if j == i else a for j, a in enumerate(at)]
        diff = (loss(*shift(1)) - loss(*shift(-1))) / 2e-5
        gg = n64(g).reshape(v.shape)
        # intermediate values are rounded to fp16, a few 2^-11 of the gradient's size each way
        assert abs(np.sum(gg * d) - diff) <= 16 * 2.0 ** -11 * np.linalg.norm(gg) * 4, i


# ------------------------------------------------------------------ gated feed-forward: a NaN in gate
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("F", [152, 150, 149])   # slopes by vectors, words and elements
def test_gated_ffn_gradient_of_a_nan_gate(act, dtype, F):
    rng = np.random.default_rng(F)
    M, D = 70, 40
    x, wg, wu = (randn(rng, s, dtype, 0.3) for s in ((M, D), (F, D), (F, D)))
    gate, up, dout = (randn(rng, (M, F), dtype) for _ in range(3))
    gate[2, 148] = float("nan")
    args = (x, wg, wu, gate, up, dout)
    made = dict(dx=torch.zeros_like(x), dw_gate=torch.zeros_like(wg), dw_up=torch.zeros_like(wu),
                dbias_gate=torch.zeros(F, device="cuda"), dbias_up=torch.zeros(F, device="cuda"))
    want = {k: torch.zeros_like(t, dtype=torch.bool) for k, t in made.items()}
    for k, row in (("dx", 2), ("dw_gate", 148), ("dw_up", 148), ("dbias_gate", 148), ("dbias_up", 148)):
        want[k][row] = True
    dit.dit_gated_ffn_backward(*args, **made, act=ACT[act])
    for k, t in made.items():
        assert torch.equal(torch.isnan(t), want[k]), k
    for k, t in made.items():
        alone = torch.zeros_like(t)
        dit.dit_gated_ffn_backward(*args, **{k: alone}, act=ACT[act])
        assert torch.equal(torch.isnan(alone), want[k]), k
    # and forward, whatever the weights of the other channels are
    wg[7, 3] = float("nan")
    for rows in (5, M):
        out = torch.zeros(rows, F, dtype=DT[dtype], device="cuda")
        dit.dit_gated_ffn_forward(x[:rows], wg, wu, out, act=ACT[act])
        assert torch.isnan(out).any(0).nonzero().flatten().tolist() == [7] and torch.isnan(out[:, 7]).all()


# widths that fill no form's threads: the first behind the one before, of several rows a warp to a whole block
@pytest.mark.parametrize("dtype,C", [*(("bf16", C) for C in (56, 248, 264, 520, 776, 1032, 1544, 2056, 4104, 8200)),
                                     *(("f32", C) for C in (28, 124, 132, 260, 388, 516, 772, 1028, 2052, 4100, 8196))])
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_reads_no_weight_behind_the_last(dtype, C, residual):
    """NaN around the weight and the rows: only what lies between them counts."""
    rng = np.random.default_rng(C)
    around = nans((3, C + 32), torch.float32)
    w = around[1, 16:16 + C]
    w.copy_(torch.from_numpy(1 + 0.3 * rng.standard_normal(C)))
    def rows():
        wide = nans((9, C + 32), DT[dtype])
        wide[1:8, 16:16 + C] = randn(rng, (7, C), dtype)
        return wide[1:8, 16:16 + C]
    x, res = rows(), rows() if residual else None
    out, q, scale = nans((7, C), DT[dtype]), torch.empty((7, C), dtype=E4M3, device="cuda"), nans((7,), torch.float32)
    dit.dit_rms_norm_forward(x, out, residual=res, weight=w)
    v = n64(x) if res is None else n64((x.float() + res.float()).to(DT[dtype]))
    ref = O.rms_norm_forward(v, n64(w))
    near(out, ref, NSTEPS * ULP * np.abs(ref), "out")
    dit.dit_rms_norm_forward(x, q, residual=res, weight=w, scale=scale)
    s = O.e4m3_scale(ref)
    near(scale, s, NSTEPS * ULP * s, "scale")
    near(q, ref / s[..., None], NSTEPS * ULP * np.abs(ref / s[..., None]), "e4m3")
    dy, dx, dw = rows(), nans((7, C), DT[dtype]), nans((C,), torch.float32)
    dit.dit_rms_norm_backward(x, dy, dx, dtotal=res, weight=w, dweight=dw)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


# ------------------------------------------------------------------ tiny and huge rows of the norm
TINY_WIDTHS = [24, 77, 255, 1536, 1535, 5000, 16384]   # several rows a warp, one, registers, rings, a whole block


def tiny_rows(rng, C, dtype):
    """Rows of 1e-39 to 1e-35, of unequal magnitudes and with zeros: their squares vanish, r is eps^-1/2.  And one of 1."""
    size = 10.0 ** np.linspace(-39, -35, 12)[:, None]
    x = rng.standard_normal((1, 12, C)) * size * 10.0 ** rng.uniform(-3, 0, (1, 12, C))
    x[rng.random(x.shape) < 0.2] = 0
    x[0, :, 0] = size[:, 0]
    x[0, 5], x[0, 8] = 0, rng.standard_normal(C)
    return torch.from_numpy(x).to(DT[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", TINY_WIDTHS)
@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("eps", [1e-6, 1e-24])
def test_rms_norm_of_tiny_rows_into_e4m3(C, dtype, affine, eps):
    rng = np.random.default_rng(C + affine)
    x = tiny_rows(rng, C, dtype)
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(C)).float().cuda() if affine else None
    q, scale = torch.empty(x.shape, dtype=E4M3, device="cuda"), nans((1, 12), torch.float32)
    dit.dit_rms_norm_forward(x, q, weight=w, scale=scale, eps=eps)
    ref = O.rms_norm_forward(n64(x), None if w is None else n64(w), eps)
    s = np.maximum(O.e4m3_scale(ref), 2.0 ** -126)   # scales are normal numbers
    near(scale, s, NSTEPS * ULP * s, "scale")
    assert scale[0, 5] == 1
    # v r is at most half a step of 2^-149 off, the weight is below 4, the scale at least 2^-126
    near(q, ref / s[..., None], NSTEPS * ULP * np.abs(ref / s[..., None]) + 2.0 ** -20, "e4m3")


@pytest.mark.parametrize("dtype,C,pad", [("bf16", 24, 0), ("f16", 77, 1), ("f32", 255, 3), ("bf16", 264, 0), ("bf16", 1536, 0), ("bf16", 1535, 1),
                                         ("f16", 5000, 8), ("f32", 8196, 0), ("bf16", 16384, 0)])
@pytest.mark.parametrize("kept", [None, "total", "x", "residual"])
@pytest.mark.parametrize("size", [1e-30, 1e38])   # v w below 2^-90, and past fp32's largest number
def test_rms_norm_of_extreme_weights_into_e4m3(dtype, C, pad, kept, size):
    """The sum comes from where it is kept, or is formed again; y itself is an ordinary number."""
    rng = np.random.default_rng(C)
    shape, scales = (2, 9, C), 10.0 ** rng.uniform(0, 4, (2, 9, 1))
    x, res = (padded(rng, shape, dtype, pad) for _ in range(2))
    x.copy_(torch.from_numpy(n64(x) * scales).to(DT[dtype]))   # r of 1 and below: v w r is finite where v w is not
    w = torch.from_numpy(rng.uniform(0.5, 1, C) * size / 8).float().cuda()
    total = {None: None, "total": padded(rng, shape, dtype, pad, fill=False), "x": x, "residual": res}[kept]
    v = n64((x.float() + res.float()).to(DT[dtype]))
    q, scale = torch.empty((2, 9, C + pad), dtype=E4M3, device="cuda")[..., pad:], nans((2, 9), torch.float32)
    dit.dit_rms_norm_forward(x, q, residual=res, total=total, weight=w, scale=scale)
    if total is not None:
        assert np.array_equal(n64(total), v)
    ref = O.rms_norm_forward(v, n64(w))
    s = O.e4m3_scale(ref)
    near(scale, s, NSTEPS * ULP * s, "scale")
    near(q, ref / s[..., None], NSTEPS * ULP * np.abs(ref / s[..., None]), "e4m3")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", TINY_WIDTHS)
def test_rms_norm_of_tiny_rows_keeps_its_digits_under_small_weights(C, dtype):
    # v w would be a subnormal number, v r and v r w are not
    rng = np.random.default_rng(C)
    x = torch.from_numpy(rng.uniform(1, 2, (2, 5, C)) * 1e-32).to(DT[dtype]).cuda()
    w = torch.from_numpy(rng.uniform(1, 2, C) * 1e-12).float().cuda()
    out = nans(x.shape, DT[dtype])
    dit.dit_rms_norm_forward(x, out, weight=w, eps=1e-24)
    ref = O.rms_norm_forward(n64(x), n64(w), 1e-24)
    near(out, ref, NSTEPS * ULP * np.abs(ref), "out")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", TINY_WIDTHS)
def test_rms_norm_of_huge_rows_is_zero_whatever_the_weight(C, dtype):
    x = torch.full((1, 3, C), 1.0, dtype=DT[dtype], device="cuda")
    x[0, 1] = 3e38
    w, out = torch.full((C,), 4.0, device="cuda"), nans((1, 3, C), DT[dtype])
    dit.dit_rms_norm_forward(x, out, weight=w)
    assert (out[0, 1] == 0).all()
    near(out[0, [0, 2]], np.full((2, C), 4 / np.sqrt(1 + 1e-6)), NSTEPS * ULP * 4)
    q, scale = torch.ones(x.shape, device="cuda").to(E4M3), nans((1, 3), torch.float32)
    dit.dit_rms_norm_forward(x, q, weight=w, scale=scale)
    assert (q[0, 1].float() == 0).all() and scale[0, 1] == 1 and (q[0, [0, 2]].float() == 448).all()


@pytest.mark.parametrize("M,D,F", [(5, 256, 40), (40, 4096, 64), (300, 256, 136), (2600, 256, 1280)])  # few rows, K split, both tiles
@pytest.mark.parametrize("bias", [False, True])
def test_gated_ffn_of_rows_with_tiny_scales(M, D, F, bias):
    """Scales whose product is no normal number where the sum times both is one."""
    rng = np.random.default_rng(M)
    x, wg, wu = (torch.from_numpy(rng.uniform(200, 448, s)).float().to(E4M3).cuda() for s in ((M, D), (F, D), (F, D)))
    xs = torch.from_numpy(rng.uniform(1, 2, M) * 2.0 ** -126).float().cuda()
    gs = torch.from_numpy(rng.uniform(1, 2, F) * 2.0 ** -22).float().cuda()
    us = torch.from_numpy(rng.uniform(1, 2, F) * 2.0 ** 88).float().cuda()
    bg, bu = (torch.from_numpy(rng.uniform(1, 2, F) * k).float().cuda() for k in (2.0 ** -126, 2.0 ** -14)) if bias else (None, None)
    out, gate, up = (nans((M, F), torch.bfloat16) for _ in range(3))
    dit.dit_gated_ffn_forward(x, wg, wu, out, gate=gate, up=up, bias_gate=bg, bias_up=bu, x_scale=xs, gate_scale=gs, up_scale=us)
    assert (gate.float() >= 2.0 ** -126).all()
    check_forward(out, gate, up, x, wg, wu, bg, bu, "silu", xs, gs, us)


def among_nans(t, left=16):
    """t in the middle of a buffer of NaN, its rows `left` elements and 24 more apart."""
    wide = nans((t.shape[0] + 2, t.shape[1] + left + 24), torch.float32).to(t.dtype) if t.dim() == 2 else nans((t.numel() + left + 24,), t.dtype)
    view = wide[1:-1, left:left + t.shape[1]] if t.dim() == 2 else wide[left:left + t.numel()]
    view.copy_(t)
    return view


@pytest.mark.parametrize("operands", ["same", "e4m3"])
@pytest.mark.parametrize("left", [16, 4, 3])   # rows of vectors, of words, of elements
@pytest.mark.parametrize("M,D,F", [(1, 72, 40), (7, 65, 33), (19, 100, 17), (32, 256, 129), (33, 72, 64), (130, 65, 67), (300, 520, 264),
                                   (40, 4096, 72), (2600, 264, 1288)])
def test_gated_ffn_reads_nothing_beside_its_operands(M, D, F, left, operands):
    rng = np.random.default_rng(M + D)
    x, wg, wu = (randn(rng, s, "bf16", 0.3) for s in ((M, D), (F, D), (F, D)))
    around = lambda t: among_nans(t, left)
    vector = lambda n, lo: around(torch.from_numpy(rng.uniform(lo, 1, n)).float().cuda())
    scales, kw = (None,) * 3, dict(bias_gate=vector(F, -1), bias_up=vector(F, -1))
    if operands == "e4m3":
        (x, xs), (wg, gs), (wu, us) = quantised(x), quantised(wg), quantised(wu)
        xs, gs, us = (among_nans(s, 0) if s.numel() == M else around(s) for s in (xs, gs, us))
        scales = xs, gs, us
        kw.update(x_scale=xs, gate_scale=gs, up_scale=us)
    x, wg, wu = around(x), around(wg), around(wu)
    out, gate, up = (torch.zeros(M, F, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    dit.dit_gated_ffn_forward(x, wg, wu, out, gate=gate, up=up, **kw)
    check_forward(out, gate, up, x, wg, wu, kw["bias_gate"], kw["bias_up"], "silu", *scales)
    if operands == "e4m3":
        return
    gate, up, dout = around(gate), around(up), around(randn(rng, (M, F), "bf16"))
    made = dict(dx=torch.zeros(M, D, dtype=torch.bfloat16, device="cuda"), dw_gate=torch.zeros(F, D, dtype=torch.bfloat16, device="cuda"),
                dw_up=torch.zeros(F, D, dtype=torch.bfloat16, device="cuda"), dbias_gate=torch.zeros(F, device="cuda"), dbias_up=torch.zeros(F, device="cuda"))
    dit.dit_gated_ffn_backward(x, wg, wu, gate, up, dout, **made)
    plain = {k: torch.zeros_like(t) for k, t in made.items()}
    alone = [t.contiguous() for t in (x, wg, wu, gate, up, dout)]
    dit.dit_gated_ffn_backward(*alone, **plain)
    for k, t in made.items():
        assert torch.equal(t, plain[k]) and torch.isfinite(t).all(), k


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [1, 7, 8, 2047, 2049, 16384, 16391, 40001])
def test_grad_norm_reads_and_writes_nothing_beside_its_tensors(dtype, n):
    rng = np.random.default_rng(n)
    for left in range(9):
        big, made = nans((n + 32,), DT[dtype]), nans((n + 32,), DT[dtype])
        g, c = big[left:left + n], made[(3 * left) % 8:][:n]
        g.copy_(torch.from_numpy(rng.standard_normal(n)))
        norm = nans((), torch.float32)
        dit.dit_grad_norm([g], norm, max_norm=0.5, clipped=[c])
        ref = O.grad_norm([n64(g)])
        assert abs(norm.item() - ref) <= 16 * ULP * ref
        near(c, n64(g) * O.clip_factor(ref, 0.5), 24 * ULP * np.abs(n64(g) * O.clip_factor(ref, 0.5)))
        assert int(torch.isnan(big).sum()) == 32 and int(torch.isnan(made).sum()) == 32
