"""Refusals of the gated feed-forward block's operators that need no GPU: the
library's checks come before any launch (pointers here are never read), and the
binding's before the library.  Workspace sizes, and views as they lie."""
import pytest
import torch

from diffusion_transformer_denoising_gb300 import dit

INVALID, SHAPE = dit.DIT_ERR_INVALID_ARG, dit.DIT_ERR_SHAPE


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(dit.LIB_PATH):
        from diffusion_transformer_denoising_gb300 import build
        build.build()
    return dit.lib()


def refused(status, call, *args, **kw):
    with pytest.raises(dit.DitError) as e:
        dit._check(call(*args, **kw) or 0)
    assert e.value.status == status, e.value
    return str(e.value)


# ------------------------------------------------------------------ rms norm
def norm_args(**kw):
    a = dict(batch=2, tokens=8, channels=16, dtype=dit.DTYPE_BF16, out_dtype=None, eps=1e-6, x=4096, xs=(128, 16), res=0,
             rs=(128, 16), total=0, ts=(128, 16), dy=0, ds=(128, 16), out=16384, os=(128, 16), scale=0, weight=0, dweight=0)
    a.update(kw)
    out_dtype = a["dtype"] if a["out_dtype"] is None else a["out_dtype"]
    return dit._NORM_ARGS.pack(a["batch"], a["tokens"], a["channels"], a["dtype"], out_dtype, a["eps"], a["x"], *a["xs"],
                               a["res"], *a["rs"], a["total"], *a["ts"], a["dy"], *a["ds"], a["out"], *a["os"],
                               a["scale"], a["weight"], a["dweight"])


E4M3 = dict(out_dtype=dit.DTYPE_E4M3, scale=32768)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(batch=1 << 20, tokens=1 << 20), SHAPE), (dict(channels=0), SHAPE),
    (dict(channels=16385), SHAPE), (dict(dtype=3), INVALID), (dict(dtype=7), INVALID), (dict(out_dtype=dit.DTYPE_F16), INVALID),
    (dict(out_dtype=9), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(x=0), INVALID), (dict(out=0), INVALID), (dict(x=4097), INVALID), (dict(scale=64), INVALID),
    (dict(E4M3, scale=0), INVALID), (dict(E4M3, scale=32770), INVALID), (dict(dy=64), INVALID), (dict(dweight=64, weight=128), INVALID),
    (dict(total=65536), INVALID),                            # the sum of one tensor
    (dict(weight=66), INVALID), (dict(xs=(-1, 16)), SHAPE), (dict(xs=(1 << 58, 16)), SHAPE), (dict(os=(128, 8)), SHAPE),
    (dict(os=(0, 16)), SHAPE), (dict(res=8192, total=65536, ts=(0, 16)), SHAPE),
    (dict(out=4096, os=(256, 32)), INVALID),                 # in place with other strides
    (dict(res=8192, total=4096, ts=(256, 32)), INVALID),
    (dict(res=8192, total=65536, out=65536), INVALID),       # two outputs in one place
    (dict(res=8192, total=4096, out=4096), INVALID),
    (dict(out=4096 + 256), INVALID),                         # over the second row of x
    (dict(E4M3, out=4096), INVALID),                         # 8 bits in place of 16
    (dict(E4M3, scale=4096), INVALID), (dict(weight=16384), INVALID), (dict(E4M3, weight=32768), INVALID),
])
def test_rms_norm_forward_refuses(L, kw, status):
    refused(status, L.dit_rms_norm_forward, norm_args(**kw), None)


def test_rms_norm_backward_refuses(L):
    g = dict(dy=65536)
    big = dict(g, weight=1024, dweight=2048)
    need = L.dit_rms_norm_workspace_bytes(norm_args(**big))
    assert need > 0 == L.dit_rms_norm_workspace_bytes(norm_args(**g))
    for kw, ws, n in ((dict(dy=0), 0, 0), (dict(g, total=8192, res=1 << 17), 0, 0), (dict(g, dweight=64), 0, 0),
                      (dict(g, **E4M3), 0, 0), (dict(g, scale=64), 0, 0), (dict(big, out=2048), 1 << 20, need),
                      (big, 0, 1 << 30), (big, 1 << 20, need - 1), (big, (1 << 20) + 8, need), (big, 16384, need),
                      (dict(big, dweight=1024), 1 << 20, need), (dict(big, dy=16384 + 32), 1 << 20, need)):
        refused(INVALID, L.dit_rms_norm_backward, norm_args(**kw), ws, n, None)
    assert L.dit_rms_norm_workspace_bytes(norm_args(channels=0, **big)) == -1


# ------------------------------------------------------------------ gated feed-forward
FWD = dict(gate=0, up=0)


def ffn_args(**kw):
    M, D, F = (kw.get(k, v) for k, v in (("rows", 64), ("width", 32), ("hidden", 48)))
    a = dict(rows=M, width=D, hidden=F, dtype=dit.DTYPE_BF16, operand=None, act=dit.ACT_SILU, reserved=0, x=1 << 20, x_s=D,
             wg=2 << 20, wg_s=D, wu=3 << 20, wu_s=D, xs=0, gs=0, us=0, bg=0, bu=0, gate=0, g_s=F, up=0, u_s=F,
             out=4 << 20, o_s=F, dx=0, dx_s=D, dwg=0, dwg_s=D, dwu=0, dwu_s=D, dbg=0, dbu=0)
    a.update(kw)
    operand = a["dtype"] if a["operand"] is None else a["operand"]
    return dit._FFN_ARGS.pack(a["rows"], a["width"], a["hidden"], a["dtype"], operand, a["act"], a["reserved"],
                              *(a[k] for k in ("x", "x_s", "wg", "wg_s", "wu", "wu_s", "xs", "gs", "us", "bg", "bu", "gate", "g_s",
                                               "up", "u_s", "out", "o_s", "dx", "dx_s", "dwg", "dwg_s", "dwu", "dwu_s", "dbg", "dbu")))


F8 = dict(operand=dit.DTYPE_E4M3, xs=4096, gs=8192, us=12288)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(width=0), SHAPE), (dict(hidden=0), SHAPE),
    (dict(width=(1 << 17) + 1), SHAPE), (dict(hidden=(1 << 17) + 1), SHAPE), (dict(rows=1 << 24, width=1 << 17), SHAPE),
    (dict(dtype=dit.DTYPE_F32), INVALID), (dict(dtype=dit.DTYPE_E4M3), INVALID), (dict(operand=dit.DTYPE_F16), INVALID),
    (dict(act=dit.ACT_NONE), INVALID), (dict(act=3), INVALID), (dict(reserved=1), INVALID), (dict(xs=4096), INVALID),
    (dict(F8, xs=0), INVALID), (dict(F8, gs=0), INVALID), (dict(F8, us=0), INVALID), (dict(F8, gs=8194), INVALID),
    (dict(dx=5 << 20), INVALID), (dict(dwg=5 << 20), INVALID), (dict(dbu=4096), INVALID), (dict(gate=5 << 20), INVALID),
    (dict(up=5 << 20), INVALID), (dict(x=0), INVALID), (dict(wg=0), INVALID), (dict(wu=0), INVALID), (dict(out=0), INVALID),
    (dict(x=(1 << 20) + 1), INVALID), (dict(x_s=-32), SHAPE), (dict(wg_s=1 << 58), SHAPE), (dict(o_s=47), SHAPE), (dict(o_s=0), SHAPE),
    (dict(out=1 << 20), INVALID),                                    # no output in place of an input
    (dict(out=(2 << 20) + 64), INVALID), (dict(gate=5 << 20, up=5 << 20), INVALID), (dict(gate=4 << 20, up=5 << 20), INVALID),
    (dict(gate=5 << 20, up=6 << 20, g_s=20), SHAPE), (dict(bg=4 << 20), INVALID), (dict(bu=4098), INVALID),
])
def test_gated_ffn_forward_refuses(L, kw, status):
    refused(status, L.dit_gated_ffn_forward, ffn_args(**kw), 64 << 20, 1 << 30, None)


BWD = dict(gate=5 << 20, up=6 << 20, dx=7 << 20, dwg=8 << 20, dwu=9 << 20, dbg=4096, dbu=8192)


@pytest.mark.parametrize("kw,status", [
    (dict(gate=0), INVALID), (dict(up=0), INVALID), (dict(gate=0, up=0), INVALID), (dict(out=0), INVALID), (dict(x=0), INVALID),
    (dict(bg=12288), INVALID), (dict(operand=dit.DTYPE_E4M3, xs=1 << 14, gs=1 << 15, us=1 << 16), INVALID), (dict(dbu=4096), INVALID),
    (dict(dx=1 << 20), INVALID), (dict(dx=5 << 20), INVALID), (dict(dwg=2 << 20), INVALID), (dict(dwg=9 << 20), INVALID),
    (dict(dwu_s=31), SHAPE), (dict(dx_s=0), SHAPE), (dict(dbg=4098), INVALID), (dict(wu=0), INVALID),
])
def test_gated_ffn_backward_refuses(L, kw, status):
    refused(status, L.dit_gated_ffn_backward, ffn_args(**{**BWD, **kw}), 64 << 20, 1 << 30, None)


def test_gated_ffn_workspace(L):
    bytes_of = lambda back=0, **kw: L.dit_gated_ffn_workspace_bytes(ffn_args(**kw), back)
    assert bytes_of(rows=0) == bytes_of(rows=1) == bytes_of(rows=8, x_s=33) == 0   # few rows are read as they lie
    assert bytes_of() == 0                                                         # whole vectors, no split of K
    # 64 rows x 32 channels in 16-byte rows
    assert bytes_of(x_s=33) == 64 * 32 * 2 and bytes_of(x=(1 << 20) + 2) == 64 * 32 * 2
    assert bytes_of(x_s=0) == 64 * 32 * 2                                          # one row for all: no matrix for the copies
    assert bytes_of(width=33, x_s=40, wg_s=40, wu_s=33) == 48 * 40 * 2
    assert bytes_of(**F8) == 0 and bytes_of(x_s=40, **F8) == 64 * 32
    assert bytes_of(1, **BWD) == 64 * 48 * 2 * 2 + 4 * 2 * 48 * 4
    assert bytes_of(1, **{**BWD, "dbg": 0, "dbu": 0}) == 64 * 48 * 2 * 2
    assert bytes_of(rows=64, width=8192, hidden=256) > 0                           # K split, sums joined in fp32
    assert bytes_of(hidden=0) == -1 and bytes_of(1, bg=64, **BWD) == -1
    for kw, ws, n in ((dict(x_s=33), 0, 1 << 30), (dict(x_s=33), 64 << 20, 4095), (dict(x_s=33), (64 << 20) + 8, 1 << 20),
                      (dict(x_s=33), 1 << 20, 1 << 20)):
        refused(INVALID, L.dit_gated_ffn_forward, ffn_args(**kw), ws, n, None)
    # the query by shapes is enough for every alignment and choice of gradients
    x, w = torch.empty(64, 32, dtype=torch.bfloat16), torch.empty(48, 32, dtype=torch.bfloat16)
    most = dit.dit_gated_ffn_workspace_bytes(x, w, backward=True)
    for k in (dict(), dict(dx=0), dict(dwg=0), dict(dwu=0), dict(dwg=0, dwu=0)):
        assert bytes_of(1, x=(1 << 20) + 2, wg_s=33, wu_s=33, **{**BWD, **k}) <= most
    assert dit.dit_gated_ffn_workspace_bytes(x, w) >= bytes_of(x_s=33, wg_s=33, wu_s=33)
    x8, w8 = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
    assert dit.dit_gated_ffn_workspace_bytes(x8, w8) == (64 + 2 * 48) * 32


def test_nothing_wanted_is_a_call_without_work(L):
    dit._check(L.dit_gated_ffn_backward(ffn_args(gate=5 << 20, up=6 << 20), 0, 0, None))
    dit._check(L.dit_gated_ffn_forward(ffn_args(rows=0, x=0, out=0), 0, 0, None))
    dit._check(L.dit_rms_norm_forward(norm_args(batch=0, x=0, out=0), None))
    dit._check(L.dit_rms_norm_forward(norm_args(tokens=0, **dict(E4M3, scale=0)), None))
    dit._check(L.dit_rms_norm_backward(norm_args(tokens=0, dy=0), 0, 0, None))


# ------------------------------------------------------------------ gradient norm
def tensors(*rows):
    import struct
    return b"".join(struct.pack("<2Qq2i", *r) for r in rows), len(rows)


BF, F32 = dit.DTYPE_BF16, dit.DTYPE_F32


@pytest.mark.parametrize("rows,max_norm,status", [
    ([(4096, 4096, -1, BF, 0)], 1.0, SHAPE), ([(4096, 4096, 1 << 45, BF, 0)], 1.0, SHAPE),
    ([(4096, 4096, 8, dit.DTYPE_E4M3, 0)], 1.0, INVALID), ([(4096, 4096, 8, 9, 0)], 1.0, INVALID), ([(4096, 4096, 8, BF, 1)], 1.0, INVALID),
    ([(0, 4096, 8, BF, 0)], 1.0, INVALID), ([(4096, 0, 8, BF, 0)], 1.0, INVALID), ([(4096, 4096, 8, BF, 0)], float("inf"), INVALID),
    ([(4097, 4097, 8, BF, 0)], 1.0, INVALID), ([(4096, 8194, 8, F32, 0)], 1.0, INVALID), ([(4096, 4096, 8, BF, 0)], -1.0, INVALID),
    ([(4096, 4096, 8, BF, 0)], float("nan"), INVALID),
    ([(4096, 4096, 8, BF, 0), (4104, 4104, 8, BF, 0)], 1.0, INVALID),       # two tensors share values
    ([(4096, 4104, 8, BF, 0)], 1.0, INVALID),                              # out over the tensor's own end
    ([(4096, 16384, 8, BF, 0), (8192, 16384, 8, BF, 0)], 1.0, INVALID),     # one out for two
    ([(4096, 8192, 8, BF, 0), (8192, 16384, 8, BF, 0)], 1.0, INVALID),      # out over the next one's gradient
    ([(1 << 20, 1 << 20, 8, BF, 0)], 1.0, INVALID), ([(256, 256, 8, F32, 0)], 1.0, INVALID),    # over the workspace, over the norm
    ([(256, 0, 8, F32, 0)], float("inf"), INVALID),                        # the norm over a gradient that is only read
])
def test_grad_norm_refuses(L, rows, max_norm, status):
    t, n = tensors(*rows)
    refused(status, L.dit_grad_norm, t, n, max_norm, 260, 1 << 20, 1 << 16, None)


def test_grad_norm_refuses_norm_and_workspace(L):
    t, n = tensors((4096, 4096, 8, BF, 0))
    need = L.dit_grad_norm_workspace_bytes(t, n)
    assert need == 8
    for norm, ws, size in ((0, 1 << 20, 8), (258, 1 << 20, 8), (256, 0, 8), (256, 1 << 20, 7), (256, (1 << 20) + 8, 8), (256, 256, 8)):
        refused(INVALID, L.dit_grad_norm, t, n, 1.0, norm, ws, size, None)
    refused(INVALID, L.dit_grad_norm, None, 1, 1.0, 256, 1 << 20, 8, None)
    refused(SHAPE, L.dit_grad_norm, t, -1, 1.0, 256, 1 << 20, 8, None)
    assert L.dit_grad_norm_workspace_bytes(t, -1) == -1
    # two gradients that are only read may share values: the same one twice
    big, k = tensors(*[(4096, 0, 1 << 30, BF, 0)] * 700)
    assert L.dit_grad_norm_workspace_bytes(big, k) == 2 * 456 * 8


# ------------------------------------------------------------------ the binding
def test_binding_refuses():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    x, y, w = bf(2, 3, 16), bf(2, 3, 16), torch.ones(16)
    fwd, bwd = dit.dit_rms_norm_forward, dit.dit_rms_norm_backward
    refused(SHAPE, fwd, x, bf(2, 3, 8))
    refused(INVALID, fwd, x, y.float())
    refused(SHAPE, fwd, x, y, weight=torch.ones(8))
    refused(INVALID, fwd, x, y, weight=w.double())
    refused(SHAPE, fwd, x, y, residual=bf(2, 3, 8), total=y)
    refused(INVALID, fwd, x, y, residual=x.float(), total=y)
    refused(SHAPE, fwd, x.transpose(1, 2), bf(2, 16, 3))
    refused(SHAPE, fwd, x, y.to(torch.float8_e4m3fn), scale=torch.ones(3, 2))
    refused(INVALID, fwd, x.double(), y.double())
    refused(SHAPE, fwd, x[0, 0, 0], y[0, 0, 0])
    refused(INVALID, fwd, x, y)                                   # not on a CUDA device
    refused(INVALID, fwd, x, y, eps="small")
    refused(SHAPE, bwd, x, bf(2, 3, 8), y)
    refused(INVALID, bwd, x, y, bf(2, 3, 16).float())
    refused(INVALID, fwd, x.float().requires_grad_(), y.float())
    refused(INVALID, fwd, x, y, weight=w.clone().requires_grad_())
    refused(INVALID, bwd, x, y.float().requires_grad_().bfloat16(), y)
    g, u = bf(6, 16), bf(5, 16)
    ffn, back = dit.dit_gated_ffn_forward, dit.dit_gated_ffn_backward
    refused(SHAPE, ffn, x, g, u, bf(2, 3, 6))
    refused(SHAPE, ffn, x, bf(6, 8), bf(6, 8), bf(2, 3, 6))
    refused(SHAPE, ffn, x, g, g.clone(), bf(2, 3, 7))
    refused(INVALID, ffn, x, g, g.half(), bf(2, 3, 6))
    refused(INVALID, ffn, x, g, g.clone(), bf(2, 3, 6).to(torch.int32))
    refused(SHAPE, ffn, x.transpose(0, 1), g, g.clone(), bf(3, 2, 6))      # rows of two strides
    refused(SHAPE, ffn, x, g, g.clone(), bf(2, 3, 6), bias_gate=torch.ones(5))
    refused(INVALID, ffn, x, g, g.clone(), bf(2, 3, 6), bias_gate=torch.ones(6).half())
    refused(INVALID, ffn, x, g, g.clone(), bf(2, 3, 6))                    # not on a CUDA device
    refused(INVALID, ffn, x, g, g.clone(), bf(2, 3, 6), act=1.5)
    refused(INVALID, ffn, x, g.float().requires_grad_().bfloat16(), g.clone(), bf(2, 3, 6))
    h = bf(2, 3, 6)
    refused(SHAPE, back, x, g, g.clone(), h, h, h, dx=bf(2, 3, 8))
    refused(INVALID, back, x, g, g.clone(), h, h, h, dw_gate=torch.ones(6, 16))
    refused(INVALID, back, x, g, g.clone(), h, h, h.float().requires_grad_().bfloat16(), dx=x)
    norm = torch.zeros(())
    one = dit.dit_grad_norm
    refused(INVALID, one, [w], norm.double())
    refused(INVALID, one, [w], torch.zeros(2))
    refused(INVALID, one, [w.double()], norm)
    refused(SHAPE, one, [torch.ones(4, 4).t()], norm)
    refused(INVALID, one, [w], norm, clipped=[w])
    refused(SHAPE, one, [w], norm, max_norm=1.0, clipped=[])
    refused(SHAPE, one, [w, None], norm, max_norm=1.0, clipped=[w, w])
    refused(SHAPE, one, [w], norm, max_norm=1.0, clipped=[torch.ones(8)])
    refused(SHAPE, one, [w], norm, max_norm=1.0, clipped=[bf(16)])
    refused(INVALID, one, [w], norm, max_norm="large")
    refused(INVALID, one, [w], norm, max_norm=float("inf"))
    refused(INVALID, one, [w.clone().requires_grad_()], norm)
    refused(INVALID, one, [w], norm)                              # not on a CUDA device


def test_views_are_read_where_they_lie():
    bf = torch.bfloat16
    t = torch.empty(3, 4, 5, 16, dtype=bf)
    p = t.data_ptr()
    assert dit._matrix("x", t, t.shape, bf) == (p, 16)
    assert dit._matrix("x", t[..., 2:10], (3, 4, 5, 8), bf) == (p + 4, 16)
    assert dit._matrix("x", t[:, 1:2, 1:2], (3, 1, 1, 16), bf) == (p + (5 + 1) * 32, 320)
    assert dit._matrix("x", t[0, 0, 0].expand(7, 16), (7, 16), bf) == (p, 0)
    assert dit._matrix("x", t[0, 0, 0], (16,), bf) == (p, 0)
    assert dit._token_view("x", t[0], (4, 5, 16), bf) == (p, 80, 16)
    assert dit._token_view("x", t[0, 0], (5, 16), bf) == (p, 0, 16)
    assert dit._token_view("x", t[0, 0, 0], (16,), bf) == (p, 0, 0)
    assert dit._token_view("x", t, t.shape, bf) == (p, 320, 16)
    assert dit._norm_rows((16,)) == (1, 1, 16) and dit._norm_rows((5, 16)) == (1, 5, 16) and dit._norm_rows((3, 4, 5, 16)) == (3, 20, 16)


def test_grad_norm_of_nothing_asks_for_some_workspace():
    assert dit.dit_grad_norm_workspace_bytes([]) == dit.dit_grad_norm_workspace_bytes([None, torch.zeros(0)]) == 8
    assert dit.dit_grad_norm_workspace_bytes([torch.zeros(2049)]) == 16


# shapes whose products split K, for one weight's gradient where they do not for two, and for neither
SPLITS = [(2048, 64, 2048), (4096, 512, 1024), (8192, 1024, 1024), (4096, 1000, 1000), (20000, 96, 96), (333, 1000, 2730),
          (64, 32, 48), (33, 4096, 64), (1 << 20, 64, 64), (1, 128, 128)]


@pytest.mark.parametrize("M,D,F", SPLITS, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_gated_ffn_workspace_by_shapes_is_enough_for_every_choice(L, M, D, F, dtype):
    x, w = torch.empty(1, dtype=dtype).expand(M, D), torch.empty(1, dtype=dtype).expand(F, D)
    most = dit.dit_gated_ffn_workspace_bytes(x, w, backward=True)
    forward = dit.dit_gated_ffn_workspace_bytes(x, w)
    code = dit.DTYPE_BF16 if dtype is torch.bfloat16 else dit.DTYPE_F16
    base, needed = dict(rows=M, width=D, hidden=F, dtype=code), 0
    for odd in (0, 1):
        views = dict(x=(1 << 20) + 2, wg_s=D + 1, wu_s=D + 1) if odd else {}
        assert L.dit_gated_ffn_workspace_bytes(ffn_args(**base, **views), 0) <= forward
        for choice in range(16):
            kept = {k: BWD[k] for i, k in enumerate(("dx", "dwg", "dwu", "dbg")) if choice >> i & 1}
            n = L.dit_gated_ffn_workspace_bytes(ffn_args(**base, **views, gate=5 << 20, up=6 << 20, **kept), 1)
            assert 0 <= n <= most, (odd, kept)
            needed = max(needed, n)
    assert needed == most


def test_clipped_entries_belong_to_the_gradients_at_their_places():
    a, b, c, d = (torch.ones(4) for _ in range(4))
    norm = torch.zeros(())
    refused(SHAPE, dit.dit_grad_norm, [None, a, b], norm, max_norm=1.0, clipped=[c, None, d])
    refused(SHAPE, dit.dit_grad_norm, [a, None], norm, max_norm=1.0, clipped=[None, c])
    refused(SHAPE, dit.dit_grad_norm, (g for g in (None, a)), norm, max_norm=1.0, clipped=(g for g in (c, None)))
    # at the same places they are taken: the next check is the device's
    assert "CUDA" in refused(INVALID, dit.dit_grad_norm, [None, a, b], norm, max_norm=1.0, clipped=[None, c, d])


def test_scales_that_require_grad_are_refused():
    x, g, u = (torch.zeros(s).to(torch.float8_e4m3fn) for s in ((3, 16), (6, 16), (6, 16)))
    out = torch.zeros(3, 6, dtype=torch.bfloat16)
    for bad in range(3):
        xs, gs, us = (torch.ones(n).requires_grad_(i == bad) for i, n in enumerate((3, 6, 6)))
        call = lambda: dit.dit_gated_ffn_forward(x, g, u, out, x_scale=xs, gate_scale=gs, up_scale=us)
        assert "requires grad" in refused(INVALID, call)
        with torch.no_grad():
            assert "CUDA" in refused(INVALID, call)


def test_forward_mode_tangents_are_refused():
    """The calls write primal values only: a tangent would be lost without a word."""
    import torch.autograd.forward_ad as fwd
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    f32 = lambda *s: torch.zeros(s)
    ffn = (bf(3, 16), bf(6, 16), bf(6, 16))
    calls = {  # inputs that a tangent may come with, and the call on them
        "rope": ([bf(1, 4, 2, 8), f32(8), bf(1, 4, 2, 8)],
                 lambda q, w, k: dit.dit_rope_forward(torch.zeros(4, 1, dtype=torch.int32), q, bf(1, 4, 2, 8), k, bf(1, 4, 2, 8),
                                                      axes=(8,), q_weight=w, k_weight=f32(8))),
        "group norm": ([bf(1, 4, 8), f32(8), f32(8)], lambda x, w, b: dit.dit_group_norm_forward(x, bf(1, 4, 8), 2, weight=w, bias=b)),
        "rms norm": ([bf(3, 16), bf(3, 16), f32(16)], lambda x, r, w: dit.dit_rms_norm_forward(x, bf(3, 16), residual=r, weight=w)),
        "rms norm gradient": ([bf(3, 16), bf(3, 16), bf(3, 16), f32(16)],
                              lambda t, dy, dt, w: dit.dit_rms_norm_backward(t, dy, bf(3, 16), dtotal=dt, weight=w)),
        "feed-forward": ([*ffn, f32(6), f32(6)],
                         lambda x, g, u, bg, bu: dit.dit_gated_ffn_forward(x, g, u, bf(3, 6), bias_gate=bg, bias_up=bu)),
        "feed-forward from e4m3": ([f32(3), f32(6), f32(6)],
                                   lambda a, b, c: dit.dit_gated_ffn_forward(*(t.to(torch.float8_e4m3fn) for t in ffn), bf(3, 6),
                                                                             x_scale=a, gate_scale=b, up_scale=c)),
        "feed-forward gradient": ([*ffn, bf(3, 6), bf(3, 6), bf(3, 6)], lambda *a: dit.dit_gated_ffn_backward(*a, dx=bf(3, 16))),
        "gradient norm": ([f32(4), bf(5)], lambda *g: dit.dit_grad_norm(list(g), torch.zeros(()))),
    }
    for name, (inputs, call) in calls.items():
        with fwd.dual_level():
            for i, t in enumerate(inputs):
                args = [fwd.make_dual(t, torch.ones_like(t)) if i == j else v for j, v in enumerate(inputs)]
                assert "tangent" in refused(INVALID, call, *args), (name, i)
                with torch.no_grad():   # which leaves tangents alone
                    assert "tangent" in refused(INVALID, call, *args), (name, i)
            assert "CUDA" in refused(INVALID, call, *inputs), name   # without one
        assert "CUDA" in refused(INVALID, call, *inputs), name
