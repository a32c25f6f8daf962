"""Refusals of the rotation and group-norm operators that need no GPU: the
library's checks come before any launch (pointers here are never read), and
the binding's before the library."""
import random

import pytest
import torch

from diffusion_transformer_denoising_gb300 import dit


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(dit.LIB_PATH):
        from diffusion_transformer_denoising_gb300 import build
        build.build()
    return dit.lib()


HEADS = dict(heads=2, reserved=0, x=4096, xs=(512, 64, 32), dy=0, ds=(0, 0, 0), out=8192, os=(512, 64, 32), weight=0,
             dweight=0)
NONE = dict(HEADS, heads=0, x=0, out=0)


def rope_args(q=HEADS, k=NONE, **kw):
    a = dict(batch=2, tokens=8, head_dim=32, dtype=dit.DTYPE_F32, style=0, n_axes=2, axes=(16, 16, 0, 0), theta=1e4,
             eps=1e-6, pos=1024, ps=(0, 2), pos_dtype=0, reserved=0)
    a.update(kw)
    heads = [v for h in (q, k) for v in (h["heads"], h["reserved"], h["x"], *h["xs"], h["dy"], *h["ds"], h["out"],
                                         *h["os"], h["weight"], h["dweight"])]
    return dit._ROPE_ARGS.pack(a["batch"], a["tokens"], a["head_dim"], a["dtype"], a["style"], a["n_axes"], *a["axes"],
                               a["theta"], a["eps"], a["pos"], *a["ps"], a["pos_dtype"], a["reserved"], *heads)


INVALID, SHAPE = dit.DIT_ERR_INVALID_ARG, dit.DIT_ERR_SHAPE


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(batch=1 << 20, tokens=1 << 20), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(head_dim=31), SHAPE), (dict(head_dim=258), SHAPE),
    (dict(dtype=3), INVALID), (dict(style=2), INVALID), (dict(pos_dtype=2), INVALID),
    (dict(n_axes=0), INVALID), (dict(n_axes=5), INVALID), (dict(axes=(15, 16, 0, 0)), INVALID),
    (dict(axes=(-2, 16, 0, 0)), INVALID), (dict(axes=(18, 16, 0, 0)), INVALID),
    (dict(theta=0.5), INVALID), (dict(theta=float("nan")), INVALID), (dict(theta=float("inf")), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(reserved=1), INVALID),
    (dict(pos=0), INVALID), (dict(pos=1026), INVALID), (dict(ps=(-16, 2)), SHAPE), (dict(ps=(0, 1 << 60)), SHAPE),
    (dict(q=NONE), SHAPE), (dict(q=dict(HEADS, heads=-1)), SHAPE), (dict(q=dict(HEADS, heads=1 << 17)), SHAPE),
    (dict(q=dict(HEADS, x=0)), INVALID), (dict(q=dict(HEADS, out=0)), INVALID), (dict(q=dict(HEADS, x=4097)), INVALID),
    (dict(q=dict(HEADS, xs=(-1, 64, 32))), SHAPE), (dict(q=dict(HEADS, xs=(1 << 58, 64, 32))), SHAPE),
    (dict(q=dict(HEADS, os=(512, 64, 31))), SHAPE),     # heads of the output overlap
    (dict(q=dict(HEADS, os=(0, 64, 32))), SHAPE),       # an expanded output
    (dict(q=dict(HEADS, os=(512, 32, 32))), SHAPE),
    (dict(q=dict(HEADS, out=4096, os=(1024, 64, 32))), INVALID),   # in place with other strides
    (dict(q=dict(HEADS, dweight=64)), INVALID), (dict(q=dict(HEADS, weight=66)), INVALID),
    (dict(k=dict(NONE, weight=64)), INVALID), (dict(k=dict(HEADS, reserved=1)), INVALID),
    (dict(k=HEADS), INVALID),                            # q and k with one output
    (dict(k=dict(HEADS, x=8192, out=12288)), INVALID),   # k read from q's output
    (dict(q=dict(HEADS, out=4096), k=dict(HEADS, out=12288)), INVALID),   # q in place of the input they share
])
def test_rope_forward_refuses(L, kw, status):
    with pytest.raises(dit.DitError) as e:
        dit._check(L.dit_rope_forward(rope_args(**kw), None))
    assert e.value.status == status, e.value


def test_rope_backward_refuses(L):
    g = dict(HEADS, dy=2048, ds=(512, 64, 32))
    many = dict(batch=1, tokens=1 << 20)
    for q, ws, n in ((dict(g, dy=0), 0, 0),                                     # no gradient
                     (dict(g, x=0, weight=64), 0, 0),                           # the norm's gradient needs x
                     (dict(g, weight=0, dweight=64), 0, 0),                     # a gradient of no weight
                     (dict(g, weight=64, dweight=128), 0, 0),                   # no workspace
                     (dict(g, weight=64, dweight=128), 1024, 16),               # too little
                     (dict(g, weight=64, dweight=128), 1032, 1 << 30)):         # not aligned
        with pytest.raises(dit.DitError) as e:
            dit._check(L.dit_rope_backward(rope_args(q=q, **many), ws, n, None))
        assert e.value.status == INVALID, e.value
    two = dict(g, weight=64, dweight=128)
    with pytest.raises(dit.DitError):
        dit._check(L.dit_rope_backward(rope_args(q=two, k=dict(two, out=16384)), 1024, 1 << 30, None))
    plain = dict(g, x=0)
    with pytest.raises(dit.DitError):                    # dk written over dq_out
        dit._check(L.dit_rope_backward(rope_args(q=plain, k=dict(plain, dy=6144, out=2048)), 0, 0, None))
    assert L.dit_rope_workspace_bytes(rope_args(q=dict(two, heads=-3))) == -1
    assert L.dit_rope_workspace_bytes(rope_args(q=two)) == 0 < L.dit_rope_workspace_bytes(rope_args(q=two, **many))


def gn_args(**kw):
    a = dict(batch=2, pixels=9, channels=12, groups=3, dtype=dit.DTYPE_F32, act=0, eps=1e-6, reserved=0, x=4096,
             xs=(108, 12), dy=0, ds=(0, 0), out=16384, os=(108, 12), weight=0, bias=0, mean=0, rstd=0, dweight=0,
             dbias=0)
    a.update(kw)
    return dit._GN_ARGS.pack(a["batch"], a["pixels"], a["channels"], a["groups"], a["dtype"], a["act"], a["eps"],
                             a["reserved"], a["x"], *a["xs"], a["dy"], *a["ds"], a["out"], *a["os"], a["weight"],
                             a["bias"], a["mean"], a["rstd"], a["dweight"], a["dbias"])


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), SHAPE), (dict(pixels=-1), SHAPE), (dict(pixels=1 << 31), SHAPE), (dict(batch=1 << 21), SHAPE),
    (dict(batch=1 << 18, pixels=1 << 20), SHAPE), (dict(channels=0), SHAPE), (dict(channels=1 << 21, groups=1), SHAPE), (dict(groups=0), SHAPE), (dict(groups=5), SHAPE),
    (dict(dtype=5), INVALID), (dict(act=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(reserved=1), INVALID), (dict(x=0), INVALID), (dict(out=0), INVALID), (dict(x=4098), INVALID),
    (dict(xs=(-1, 12)), SHAPE), (dict(os=(0, 12)), SHAPE), (dict(os=(108, 11)), SHAPE), (dict(os=(12, 12)), SHAPE),
    (dict(out=4096, os=(216, 24)), INVALID), (dict(dweight=64, weight=128), INVALID), (dict(dbias=64, bias=128), INVALID),
    (dict(mean=64, rstd=64), INVALID), (dict(weight=66), INVALID),
])
def test_group_norm_forward_refuses(L, kw, status):
    with pytest.raises(dit.DitError) as e:
        dit._check(L.dit_group_norm_forward(gn_args(**kw), 1024, 1 << 30, None))
    assert e.value.status == status, e.value


def test_group_norm_refuses_bad_workspace_and_missing_statistics(L):
    big = dict(pixels=1 << 20, xs=(12 << 20, 12), os=(12 << 20, 12))
    need = L.dit_group_norm_workspace_bytes(gn_args(**big), 0)
    assert need > 0
    for ws, n in ((0, 1 << 40), (1024, need - 1), (1032, need)):
        with pytest.raises(dit.DitError) as e:
            dit._check(L.dit_group_norm_forward(gn_args(**big), ws, n, None))
        assert e.value.status == INVALID
    back = dict(dy=2048, ds=(108, 12))
    for kw in (dict(mean=64), dict(rstd=64), dict(mean=64, rstd=128, dy=0), dict(mean=64, rstd=128, dweight=256),
               dict(mean=64, rstd=128, weight=192, bias=224, dweight=256, dbias=256)):
        with pytest.raises(dit.DitError) as e:
            dit._check(L.dit_group_norm_backward(gn_args(**{**back, **kw}), 1024, 1 << 30, None))
        assert e.value.status == INVALID
    assert L.dit_group_norm_workspace_bytes(gn_args(groups=5), 1) == -1


def test_empty_calls_are_no_ops(L):
    dit._check(L.dit_rope_forward(rope_args(tokens=0, pos=0, q=dict(HEADS, x=0, out=0)), None))
    dit._check(L.dit_group_norm_forward(gn_args(batch=0, x=0, out=0), 0, 0, None))


def test_binding_refuses():
    z = torch.zeros
    pos, q = z(8, 2, dtype=torch.int32), z(2, 8, 3, 32)
    ok = dict(axes=(16, 16))
    for status, pos_, q_, out, kw in (
            (INVALID, pos, q, q, ok),                                       # host tensors
            (SHAPE, pos, q[0], q[0], ok), (SHAPE, pos[:7], q, q, ok), (SHAPE, pos[:, :1], q, q, ok),
            (INVALID, pos.long(), q, q, ok), (INVALID, pos, q, q.bfloat16(), ok), (SHAPE, pos, q, q[:, :, :2], ok),
            (SHAPE, pos, q, z(2, 8, 3, 64)[..., ::2], ok), (INVALID, pos, q.double(), q.double(), ok),
            (INVALID, pos, q, q, dict(axes=())), (INVALID, pos, q, q, dict(axes=(8,) * 5)),
            (INVALID, pos, q, q, dict(ok, q_weight=z(32, dtype=torch.bfloat16))), (SHAPE, pos, q, q, dict(ok, q_weight=z(31))),
            (INVALID, pos, q, q, dict(ok, k=q))):
        with pytest.raises(dit.DitError) as e:
            dit.dit_rope_forward(pos_, q_, out, **kw)
        assert e.value.status == status, (e.value, pos_.shape, kw)
    x = z(2, 4, 5, 12)
    for status, x_, y, kw in ((INVALID, x, x, {}), (SHAPE, x[0, 0], x[0, 0], {}), (SHAPE, x, x[:, :3], {}),
                              (SHAPE, z(2, 12, 4, 5).permute(0, 2, 3, 1), z(2, 12, 4, 5).permute(0, 2, 3, 1), {}),
                              (SHAPE, x, z(2, 4, 7, 12)[:, :, :5], {}), (INVALID, x, x.half(), {}),
                              (SHAPE, x, x, dict(weight=z(11))), (SHAPE, x, x, dict(mean=z(2, 4))),
                              (INVALID, x, x, dict(bias=z(12, dtype=torch.int32)))):
        with pytest.raises(dit.DitError) as e:
            dit.dit_group_norm_forward(x_, y, 3, **kw)
        assert e.value.status == status, (e.value, x_.shape, kw)


def test_workspace_sizes():
    assert dit.dit_rope_workspace_bytes(128) >= 128 * 4
    with pytest.raises(dit.DitError):
        dit.dit_rope_workspace_bytes(257)
    x = torch.zeros(2, 8, 8, 64)
    for backward in (False, True):
        assert dit.dit_group_norm_workspace_bytes(x, 32, backward) >= 0
    with pytest.raises(dit.DitError):
        dit.dit_group_norm_workspace_bytes(x, 48, False)


def test_pixel_views_are_read_where_they_lie():
    """Middle axes of any strides, expanded ones (stride 0) among them: either the binding's one pixel stride reaches
    exactly the view's elements, or the view is refused."""
    rng = random.Random(1)
    taken = refused = 0
    for _ in range(3000):
        shape = [rng.choice([1, 1, 2, 3]) for _ in range(rng.choice([3, 4, 4, 5]))] + [rng.choice([1, 4])]
        t = torch.arange(4096.0)
        stride, span = [0] * len(shape), 1
        for a in rng.sample(range(len(shape)), len(shape)) if rng.random() < 0.2 else reversed(range(len(shape))):
            stride[a] = 0 if a < len(shape) - 1 and rng.random() < 0.3 else span
            span = max(span, stride[a] * shape[a]) + (rng.choice([0, 0, 0, 2]) if a < len(shape) - 1 else 0)
        if shape[-1] > 1 and stride[-1] != 1:
            continue
        v = t.as_strided(shape, stride)
        try:
            ptr, sb, step = dit._pixel_view("x", v, v.shape, v.dtype)
        except dit.DitError as e:
            assert e.status == SHAPE
            refused += 1
            continue
        assert ptr == v.data_ptr()
        pixels = v.reshape(shape[0], -1, shape[-1])
        assert torch.equal(pixels, t.as_strided(pixels.shape, (sb, step, 1))), (shape, stride)
        taken += 1
    assert taken > 500 and refused > 100
    # an image whose rows are one row repeated has two pixel strides, in either order of the axes
    row, col = torch.zeros(2, 1, 5, 12), torch.zeros(2, 4, 1, 12)
    dense = torch.zeros(2, 4, 5, 12)
    for wide in (row.expand(2, 4, 5, 12), col.expand(2, 4, 5, 12)):
        for x, y in ((wide, dense), (dense, wide)):
            with pytest.raises(dit.DitError) as e:
                dit.dit_group_norm_forward(x, y, 3)
            assert e.value.status == SHAPE, e.value
    every = torch.zeros(2, 1, 1, 12).expand(2, 4, 5, 12)      # one pixel for all: one stride, 0
    assert dit._pixel_view("x", every, every.shape, every.dtype)[2] == 0


BACK = dict(HEADS, dy=2**20, ds=(512, 64, 32), weight=2**21, dweight=2**22)


@pytest.mark.parametrize("call,kw", [
    ("rope", dict(q=dict(HEADS, out=4096 + 64))),                                    # part of a row further on
    ("rope", dict(q=HEADS, k=dict(HEADS, x=4096 + 2048, out=8192 + 2048))),          # half of q's output
    ("rope", dict(q=dict(HEADS, weight=8192 + 3968))),                               # a weight under the output's last row
    ("rope", dict(pos=8192 + 64)),
    ("rope_backward", dict(q=dict(BACK, dweight=BACK["weight"]))),                   # a weight's gradient over the weight
    ("rope_backward", dict(q=dict(BACK, dweight=BACK["weight"] + 64))),
    ("rope_backward", dict(q=dict(BACK, dweight=BACK["dy"] + 128))),
    ("rope_backward", dict(q=BACK, k=dict(BACK, dy=2**23, out=2**24, weight=2**25, dweight=BACK["dweight"] + 124))),
    ("rope_backward", dict(q=dict(BACK, dweight=0), k=dict(BACK, dy=2**23, out=2**24, weight=2**25, dweight=BACK["weight"]))),
    ("rope_backward", dict(tokens=1 << 20, batch=1, q=dict(BACK, xs=(0, 0, 32), ds=(0, 0, 32), os=(0, 64, 32), out=2**40,
                                                         dweight=2**30 + 64))),      # inside the workspace
    ("gn", dict(out=4096 + 48)), ("gn", dict(mean=4096)), ("gn", dict(weight=2048, rstd=2048)),
    ("gn", dict(mean=64, rstd=84)), ("gn", dict(bias=16384 + 860, weight=128)),
    ("gn_backward", dict(weight=2048, dweight=2048)), ("gn_backward", dict(bias=2048, dbias=2092)),
    ("gn_backward", dict(weight=2048, dweight=512)), ("gn_backward", dict(weight=2048, dweight=536)),   # over mean, over rstd
    ("gn_backward", dict(out=2**20 + 4)), ("gn_backward", dict(weight=2048, bias=2096, dweight=1024, dbias=1068)),
])
def test_outputs_that_meet_anything_else_are_refused(L, call, kw):
    ws = 2**30, 2**20
    with pytest.raises(dit.DitError) as e:
        if call == "rope":
            dit._check(L.dit_rope_forward(rope_args(**kw), None))
        elif call == "rope_backward":
            dit._check(L.dit_rope_backward(rope_args(**kw), *ws, None))
        elif call == "gn":
            dit._check(L.dit_group_norm_forward(gn_args(**kw), *ws, None))
        else:
            kw = {**dict(dy=2**20, ds=(108, 12), mean=512, rstd=536), **kw}
            dit._check(L.dit_group_norm_backward(gn_args(**kw), *ws, None))
    assert e.value.status == INVALID and "overlaps" in str(e.value), e.value


def test_views_of_one_buffer_pass_where_they_do_not_meet(L):
    """The library's answer against the sets of elements, for pairs of views laid into one buffer in every order."""
    import itertools
    rng = random.Random(2)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        batch, pixels, channels = rng.choice([1, 2, 3]), rng.choice([1, 3, 4]), rng.choice([3, 6])
        base = rng.choice([channels, 2 * channels, 3 * channels, channels + 1])

        def strides(free):
            if free and rng.random() < 0.3:
                return rng.choice([0, 1, channels, base]), rng.choice([0, 1, channels])
            inner, outer = base, base * pixels + rng.choice([0, 0, channels, 1])
            return (outer, inner) if rng.random() < 0.5 else (inner, base * batch + rng.choice([0, 0, channels]))

        xs, os = strides(True), strides(False)
        x, out = 4096 * 16, 4096 * 16 + 4 * rng.randint(-60, 60)
        at = lambda p, st: {p // 4 + b * st[0] + i * st[1] + c for b, i, c in
                            itertools.product(range(batch), range(pixels), range(channels))}
        used = [s for n, s in zip((batch, pixels), os) if n > 1]
        status = L.dit_group_norm_forward(gn_args(batch=batch, pixels=pixels, channels=channels, groups=1, x=x, xs=xs,
                                                  out=out, os=os), 2**30, 2**20, None)
        message = L.dit_last_error().decode()
        if status == SHAPE:
            assert len(at(out, os)) < batch * pixels * channels or used
            continue
        same = x == out and all(n == 1 or a == b for n, a, b in zip((batch, pixels), xs, os))
        if x == out and not same:
            assert status == INVALID
            continue
        meets = not same and bool(at(x, xs) & at(out, os))
        assert ("overlaps" in message) == meets, (message, batch, pixels, channels, x, xs, out, os)
        seen[meets] += 1
    assert min(seen.values()) > 300, seen
    # q and k of a packed projection written over themselves, and a large buffer's slices in any order
    for step, heads in ((3, 0), (1, 1)):
        H, d, N = 4, 32, 1 << 20
        st = (N * 3 * H * d, 3 * H * d, d) if step == 3 else (3 * N * H * d, d, N * d)
        off = H * d * 4 if step == 3 else H * N * d * 4
        h = lambda i: dict(HEADS, heads=H, x=2**40 + i * off, out=2**40 + i * off, xs=st, os=st)
        status = L.dit_rope_forward(rope_args(tokens=N, q=h(0), k=h(1), pos=2**20), None)
        assert status != dit.DIT_OK and "overlaps" not in L.dit_last_error().decode()
        status = L.dit_rope_forward(rope_args(tokens=N, q=h(0), k=dict(h(1), out=h(0)["out"] + 64), pos=2**20), None)
        assert status == INVALID and "overlaps" in L.dit_last_error().decode()


def test_tensors_that_require_grad_are_refused_unless_grad_mode_is_off():
    z = torch.zeros
    pos, q, w = z(8, 2, dtype=torch.int32), z(2, 8, 3, 32), z(32)
    x, st, c = z(2, 5, 12), z(2, 3), z(12)
    calls = [lambda q, w, x, st, c: dit.dit_rope_forward(pos, q, q, axes=(16, 16), q_weight=w),
             lambda q, w, x, st, c: dit.dit_rope_backward(pos, q, q, axes=(16, 16), q=q, q_weight=w, dq_weight=z(32)),
             lambda q, w, x, st, c: dit.dit_group_norm_forward(x, x, 3, weight=c, bias=c),
             lambda q, w, x, st, c: dit.dit_group_norm_backward(x, x, st, st.clone(), x, 3, weight=c)]
    for n, call in enumerate(calls):
        args = (q, w, x, st, c)
        for i in (0, 1) if n < 2 else (2, 4):
            with_grad = list(args)
            with_grad[i] = args[i].clone().requires_grad_()
            with pytest.raises(dit.DitError) as e:
                call(*with_grad)
            assert e.value.status == INVALID and "autograd" in str(e.value)
            with torch.no_grad(), pytest.raises(dit.DitError) as e:      # refused for its device only
                call(*with_grad)
            assert "CUDA" in str(e.value)
    at = z(8, 2, requires_grad=True)                                      # learnt positions have no gradient here
    with pytest.raises(dit.DitError) as e:
        dit.dit_rope_forward(at, q, q, axes=(16, 16))
    assert "autograd" in str(e.value)
    seen = []

    class Turn(torch.autograd.Function):                                 # how a program gives the operator to autograd
        @staticmethod
        def forward(ctx, q):
            seen.append(torch.is_grad_enabled())
            with pytest.raises(dit.DitError) as e:
                calls[0](q, w, x, st, c)
            assert "CUDA" in str(e.value)
            return q * 2

        @staticmethod
        def backward(ctx, dy):
            seen.append(torch.is_grad_enabled())
            return dy

    Turn.apply(q.clone().requires_grad_()).sum().backward()
    assert seen == [False, False]


def test_workspace_sizes_follow_the_restated_plan():
    """Also pins down that only sizes and type count: the query's answer is enough for any strides and alignment."""
    from tests import group_norm_plan as G
    rng = random.Random(3)
    forms = set()
    for _ in range(3000):
        groups = rng.choice([1, 2, 3, 4, 8, 13, 32])
        channels = groups * rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 40, 300])
        batch, pixels = int(2 ** rng.uniform(0, 6)), int(2 ** rng.uniform(0, 20))
        dtype, backward = rng.choice([dit.DTYPE_F32, dit.DTYPE_BF16]), rng.random() < 0.5
        elem = 4 if dtype == dit.DTYPE_F32 else 2
        got = dit.lib().dit_group_norm_workspace_bytes(
            gn_args(batch=batch, pixels=pixels, channels=channels, groups=groups, dtype=dtype, x=rng.randint(0, 1 << 20),
                    xs=(rng.randint(0, 99), rng.randint(0, 99))), backward)
        want = G.workspace(batch, pixels, channels, groups, elem, backward)
        assert got == want, (batch, pixels, channels, groups, dtype, backward)
        p = G.plan(batch, pixels, channels, groups, elem, 1, backward)
        forms.add((p["cluster"], p["whole_batch"], p["unit"] == 1))
    assert len(forms) >= 4


def test_workspace_query_of_a_tensor_that_requires_grad():
    x = torch.zeros(2, 8, 8, 64, requires_grad=True)
    assert dit.dit_group_norm_workspace_bytes(x, 32, True) == dit.dit_group_norm_workspace_bytes(x.detach(), 32, True)


def test_scalars_that_the_structures_cannot_hold_are_refused():
    pos, q, x = torch.zeros(8, 2, dtype=torch.int32), torch.zeros(2, 8, 3, 32), torch.zeros(2, 5, 12)
    for kw in (dict(axes=(16.0, 16)), dict(axes=(2**40, 16)), dict(axes=(16, 16), theta=1e39), dict(axes=(16, 16), eps="1"),
               dict(axes=(16, 16), style=2**31), dict(axes=(16, 16), style="split")):
        with pytest.raises(dit.DitError) as e:
            dit.dit_rope_forward(pos, q, q, **kw)
        assert e.value.status == INVALID
    for groups, kw in ((3.0, {}), (2**33, {}), (3, dict(eps=1e40)), (3, dict(act="silu"))):
        with pytest.raises(dit.DitError) as e:
            dit.dit_group_norm_forward(x, x, groups, **kw)
        assert e.value.status == INVALID
    for call in (lambda: dit.dit_rope_workspace_bytes(2**40), lambda: dit.dit_group_norm_workspace_bytes(x, 2**33, True)):
        with pytest.raises(dit.DitError) as e:
            call()
        assert e.value.status in (INVALID, SHAPE)
