"""The RMS norm with the residual's addition, the gated feed-forward and the
gradient norm, as cases to be measured.

Three operators of the feed-forward half of a transformer block:

* norm: the residual's addition and an RMS norm over channels, with an output
  in the type of the input or in e4m3 with a scale for each row; its gradient;
* ffn: both projections of a gated feed-forward, the activation and the
  product, in bf16, fp16 or from e4m3 operands with scales; its gradient;
* clip: the norm of all gradients of a model together, and their clipping.

`run` makes the framework's calls where `own` is true and computes the plain
form (elementary torch operations, 32 bits, rounded once) where it is false.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def _norm(name, dtype, batch, tokens, channels, residual=True, out="same", affine=True, backward=False, pad=0):
    """out: same = the input's type; e4m3 = 8 bits with a scale for each row.
    pad: channels between one row's and the next's (a slice of a wider buffer)."""
    return dict(name=name, op="norm", dtype=dtype, batch=batch, tokens=tokens, channels=channels, residual=residual,
                out=out, affine=affine, backward=backward, pad=pad)


def _ffn(name, dtype, tokens, width, hidden, act="silu", operands="same", bias=False, saved=False, backward=False,
         packed=False):
    """operands: same = of the output's type; e4m3 = 8 bits with scales per token and per output channel.
    saved: the forward pass keeps what the gradient needs.  packed: both weights are halves of one tensor."""
    return dict(name=name, op="ffn", dtype=dtype, tokens=tokens, width=width, hidden=hidden, act=act,
                operands=operands, bias=bias, saved=saved, backward=backward, packed=packed)


def _clip(name, blocks, width, hidden, vectors, large=1.0, clipped=True):
    """Gradients of `blocks` blocks: two bf16 matrices [hidden, width] and `vectors` fp32 vectors of `width` each.
    large: their typical size; clipped: whether their norm is above the limit."""
    return dict(name=name, op="clip", blocks=blocks, width=width, hidden=hidden, vectors=vectors, large=large,
                clipped=clipped)


def listed():
    return [
        # one token of a video model's width: nothing but latency
        _norm("norm_one_token", "bf16", 1, 1, 1536),
        # 81 frames of 480x832 as 32760 tokens, conditional and unconditional pass of one step
        _norm("norm_video_pair", "bf16", 2, 32760, 1536),
        # the same tokens on their way into an 8-bit projection
        _norm("norm_video_e4m3", "bf16", 1, 32760, 1536, out="e4m3"),
        # fine-tuning the video model: the gradient of both addends and of the weight
        _norm("norm_video_grad", "bf16", 1, 32760, 1536, backward=True),
        # 32 bits, odd rows in a slice of a wider buffer, no residual
        _norm("norm_odd_grad", "f32", 3, 1237, 1001, residual=False, backward=True, pad=3),
        # one token through both projections of the video model's width: the weights are all there is to read
        _ffn("ffn_one_token", "bf16", 1, 1536, 8960),
        # the video model's tokens, serving
        _ffn("ffn_video", "bf16", 32760, 1536, 8960),
        # the same from 8-bit operands
        _ffn("ffn_video_e4m3", "bf16", 32760, 1536, 8960, operands="e4m3"),
        # fine-tuning: the gradients of a quarter of the video tokens
        _ffn("ffn_video_grad", "bf16", 8190, 1536, 8960, backward=True),
        # a small ragged batch of condition tokens; sizes that fill no tile, with biases, weights packed in one
        _ffn("ffn_odd_grad", "f16", 333, 1000, 2730, act="gelu", bias=True, packed=True, backward=True),
        # the norm weights and biases of a small model: latency
        _clip("clip_small", 2, 128, 512, 6),
        # the feed-forward weights and vectors of the whole video model
        _clip("clip_video", 30, 1536, 8960, 6),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.random()
    if kind < 0.4:
        channels = _log_int(rng, 16, 8192)
        if rng.random() < 0.75:
            channels = max(8, channels // 8 * 8)
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        backward = rng.random() < 0.4
        batch = rng.choice([1, 1, 2, 3])
        tokens = _log_int(rng, 1, max(1, min(70000, 400_000_000 // (batch * channels * (4 if dtype == "f32" else 2)))))
        case = _norm("", dtype, batch, tokens, channels, residual=rng.random() < 0.7,
                     out=rng.choice(["same", "e4m3"]) if not backward else "same", affine=rng.random() < 0.85,
                     backward=backward, pad=rng.choice([0, 0, 0, 8, 5]))
    elif kind < 0.8:
        backward = rng.random() < 0.4
        operands = "e4m3" if not backward and rng.random() < 0.35 else "same"
        step = rng.choice([1, 8, 16, 64, 64, 128])
        width, hidden = (max(step, v // step * step) for v in (_log_int(rng, 64, 4096), _log_int(rng, 64, 12288)))
        most = int(1.8e12 / (4 * width * hidden * (2 if backward else 1)))
        tokens = _log_int(rng, 1, max(1, min(40000, most)))
        case = _ffn("", rng.choice(["bf16", "bf16", "f16"]), tokens, width, hidden, act=rng.choice(["silu", "gelu"]),
                    operands=operands, bias=rng.random() < 0.3, saved=operands == "same" and rng.random() < 0.4,
                    backward=backward, packed=rng.random() < 0.3)
    else:
        width, hidden = _log_int(rng, 32, 2048), _log_int(rng, 64, 8960)
        blocks = _log_int(rng, 1, max(1, min(60, 800_000_000 // (2 * width * hidden))))
        case = _clip("", blocks, width, hidden, rng.choice([0, 1, 2, 6, 9]), large=rng.choice([1.0, 1e-4, 1e3]),
                     clipped=rng.random() < 0.75)
    return {k: v for k, v in case.items() if k != "name"}


# ------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(shape, dtype=torch.float32, device="cuda", generator=g)


def _quantised(x):
    """e4m3 values and the scale of each row."""
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    return (x / scale[:, None]).to(_E4M3), scale


def _prepare_norm(case, g):
    B, N, C, t = case["batch"], case["tokens"], case["channels"], _DTYPES[case["dtype"]]
    s = {"case": case}

    def rows(fill=True):
        v = torch.empty((B, N, C + case["pad"]), dtype=t, device="cuda")
        if fill:
            v.copy_(_randn(g, *v.shape))
        return v[..., :C]

    s["w"] = 1 + 0.2 * _randn(g, C) if case["affine"] else None
    if case["backward"]:
        s["total"], s["dout"], s["dx"] = rows(), rows(), torch.empty((B, N, C), dtype=t, device="cuda")
        s["dtotal"] = rows() if case["residual"] else None
        s["dw"] = torch.empty(C, device="cuda") if case["affine"] else None
        return s
    s["x"] = rows()
    s["residual"] = rows().mul_(4) if case["residual"] else None
    s["total"] = rows(False) if case["residual"] else None
    s["out"] = torch.empty((B, N, C), dtype=_E4M3 if case["out"] == "e4m3" else t, device="cuda")
    s["scale"] = torch.empty((B, N), device="cuda") if case["out"] == "e4m3" else None
    return s


def _prepare_ffn(case, g):
    M, D, F, t = case["tokens"], case["width"], case["hidden"], _DTYPES[case["dtype"]]
    s = {"case": case}
    x, both = _randn(g, M, D), _randn(g, 2 * F, D) / math.sqrt(D)
    s["xs"] = s["gs"] = s["us"] = None
    if case["operands"] == "e4m3":
        s["x"], s["xs"] = _quantised(x)
        both, scales = _quantised(both)
        s["gs"], s["us"] = scales[:F], scales[F:]
    else:
        s["x"], both = x.to(t), both.to(t)
    del x
    s["wg"], s["wu"] = (both[:F], both[F:]) if case["packed"] else (both[:F].clone(), both[F:].clone())
    s["bg"], s["bu"] = (0.3 * _randn(g, 2, F)).unbind() if case["bias"] else (None, None)
    s["g"] = s["u"] = None
    if case["backward"]:
        # what the forward pass left behind
        s["g"], s["u"] = (_pre(s["x"], s[w], s[b]).to(t) for w, b in (("wg", "bg"), ("wu", "bu")))
        s["dout"] = _randn(g, M, F).to(t)
        s["dx"], s["dwg"], s["dwu"] = torch.empty_like(s["x"]), torch.empty_like(s["wg"]), torch.empty_like(s["wu"])
        s["dbg"], s["dbu"] = torch.empty(2, F, device="cuda").unbind() if case["bias"] else (None, None)
        return s
    s["out"] = torch.empty((M, F), dtype=t, device="cuda")
    if case["saved"]:
        s["g"], s["u"] = torch.empty_like(s["out"]), torch.empty_like(s["out"])
    return s


def _prepare_clip(case, g):
    W, H, V = case["width"], case["hidden"], case["vectors"]
    n = 2 * case["blocks"]
    s = {"case": case}
    # gradients as a program keeps them: parts of one buffer for each type
    s["matrices"] = (_randn(g, n * H * W) * case["large"]).to(torch.bfloat16)
    s["vectors"] = _randn(g, case["blocks"] * V * W) * case["large"]
    s["new_matrices"], s["new_vectors"] = torch.empty_like(s["matrices"]), torch.empty_like(s["vectors"])

    def parts(matrices, vectors):
        return [*matrices.view(n, H, W).unbind(), *vectors.view(-1, W).unbind()]

    s["grads"], s["outs"] = parts(s["matrices"], s["vectors"]), parts(s["new_matrices"], s["new_vectors"])
    norm = case["large"] * math.sqrt(n * H * W + case["blocks"] * V * W)
    s["limit"] = norm * (0.37 if case["clipped"] else 2.0)
    s["norm"] = torch.empty((), device="cuda")
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return {"norm": _prepare_norm, "ffn": _prepare_ffn, "clip": _prepare_clip}[case["op"]](case, g)


# ------------------------------------------------------------------ plain forms
def _pre(x, w, b):
    v = x.float() @ w.float().t()
    return v if b is None else v + b


def _act(name, v):
    if name == "silu":
        return v * torch.sigmoid(v)
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))


def _act_and_slope(name, v):
    if name == "silu":
        sig = torch.sigmoid(v)
        return v * sig, sig * (1 + v * (1 - sig))
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (v + 0.044715 * v * v * v))
    return 0.5 * v * (1 + th), 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * c * (1 + 3 * 0.044715 * v * v)


def _plain_norm(s):
    c, w = s["case"], s["w"]
    if c["backward"]:
        v, dy = s["total"].float(), s["dout"].float()
        r = torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)
        t = v * r
        g = dy if w is None else dy * w
        dx = r * (g - t * (g * t).mean(-1, keepdim=True))
        if s["dtotal"] is not None:
            dx = dx + s["dtotal"].float()
        dx = dx.to(s["dout"].dtype)
        return [dx] if w is None else [dx, (dy * t).sum((0, 1))]
    total = s["x"]
    if s["residual"] is not None:
        total = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    v = total.float()
    y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)
    if w is not None:
        y = y * w
    out = [total] if s["residual"] is not None else []
    if c["out"] == "same":
        return out + [y.to(s["x"].dtype)]
    q, scale = _quantised(y.flatten(0, 1))
    return out + [q.view(y.shape), scale.view(y.shape[:-1])]


def _scaled(q, scale):
    return q if scale is None else q.float() * scale[:, None]


def _plain_ffn(s):
    c, t = s["case"], _DTYPES[s["case"]["dtype"]]
    if c["backward"]:
        a, slope = _act_and_slope(c["act"], s["g"].float())
        dh = s["dout"].float()
        du, dg = dh * a, dh * s["u"].float() * slope
        x = s["x"].float()
        dx = dg @ s["wg"].float() + du @ s["wu"].float()
        out = [dx.to(t), (dg.t() @ x).to(t), (du.t() @ x).to(t)]
        return out + [dg.sum(0), du.sum(0)] if c["bias"] else out
    x = _scaled(s["x"], s["xs"])
    g, u = _pre(x, _scaled(s["wg"], s["gs"]), s["bg"]), _pre(x, _scaled(s["wu"], s["us"]), s["bu"])
    h = (_act(c["act"], g) * u).to(t)
    return [h, g.to(t), u.to(t)] if c["saved"] else [h]


def _plain_clip(s):
    square = [v.float().view(-1, s["case"]["width"]).square().sum(-1).double().sum()
              for v in (s["matrices"], s["vectors"])]
    norm = (square[0] + square[1]).sqrt().float()
    factor = torch.where(norm > s["limit"], s["limit"] / norm, torch.ones_like(norm))
    return [norm, (s["matrices"].float() * factor).to(torch.bfloat16), s["vectors"] * factor]


# ------------------------------------------------------------------ the framework's calls
def _own_norm(s):
    from diffusion_transformer_denoising_gb300 import dit

    if s["case"]["backward"]:
        dit.dit_rms_norm_backward(s["total"], s["dout"], s["dx"], dtotal=s["dtotal"], weight=s["w"], dweight=s["dw"],
                                  eps=1e-6)
        return [s["dx"]] if s["w"] is None else [s["dx"], s["dw"]]
    dit.dit_rms_norm_forward(s["x"], s["out"], residual=s["residual"], total=s["total"], weight=s["w"],
                             scale=s["scale"], eps=1e-6)
    return [v for v in (s["total"], s["out"], s["scale"]) if v is not None]


def _own_ffn(s):
    from diffusion_transformer_denoising_gb300 import dit

    c = s["case"]
    act = dit.ACT_SILU if c["act"] == "silu" else dit.ACT_GELU
    if c["backward"]:
        dit.dit_gated_ffn_backward(s["x"], s["wg"], s["wu"], s["g"], s["u"], s["dout"], dx=s["dx"], dw_gate=s["dwg"],
                                   dw_up=s["dwu"], dbias_gate=s["dbg"], dbias_up=s["dbu"], act=act)
        return [v for v in (s["dx"], s["dwg"], s["dwu"], s["dbg"], s["dbu"]) if v is not None]
    dit.dit_gated_ffn_forward(s["x"], s["wg"], s["wu"], s["out"], gate=s["g"], up=s["u"], bias_gate=s["bg"],
                              bias_up=s["bu"], x_scale=s["xs"], gate_scale=s["gs"], up_scale=s["us"], act=act)
    return [s["out"], s["g"], s["u"]] if c["saved"] else [s["out"]]


def _own_clip(s):
    from diffusion_transformer_denoising_gb300 import dit

    dit.dit_grad_norm(s["grads"], s["norm"], max_norm=s["limit"], clipped=s["outs"])
    return [s["norm"], s["new_matrices"], s["new_vectors"]]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "ffn": _own_ffn, "clip": _own_clip}[op](state)
    return {"norm": _plain_norm, "ffn": _plain_ffn, "clip": _plain_clip}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        e = 4 if case["dtype"] == "f32" else 2
        rows, C = case["batch"] * case["tokens"], case["channels"]
        w = 4 * C if case["affine"] else 0
        if case["backward"]:
            return {"bytes": rows * C * e * (4 if case["residual"] else 3) + 2 * w, "flops": 11 * rows * C}
        out = rows * C + 4 * rows if case["out"] == "e4m3" else rows * C * e
        return {"bytes": rows * C * e * (3 if case["residual"] else 1) + out + w, "flops": 5 * rows * C}
    if case["op"] == "ffn":
        M, D, F = case["tokens"], case["width"], case["hidden"]
        e = 1 if case["operands"] == "e4m3" else 2
        bias = 8 * F if case["bias"] else 0
        if case["backward"]:
            return {"bytes": 2 * (2 * M * D + 4 * F * D + 3 * M * F) + bias, "flops": 8 * M * D * F}
        out = 2 * M * F * (3 if case["saved"] else 1)
        return {"bytes": e * (M * D + 2 * F * D) + out + bias + (4 * (M + 2 * F) if e == 1 else 0),
                "flops": 4 * M * D * F}
    W, H, n = case["width"], case["hidden"], case["blocks"]
    matrices, vectors = 2 * n * H * W, n * case["vectors"] * W
    return {"bytes": 2 * (2 * matrices + 4 * vectors) + 4, "flops": 3 * (matrices + vectors)}


# ------------------------------------------------------------------ 64 bits
def _exact_norm(s):
    c, w = s["case"], s["w"]
    if c["backward"]:
        v = s["total"].double().requires_grad_()
        w = None if w is None else w.double().requires_grad_()
        y = v / torch.sqrt(torch.linalg.vector_norm(v, dim=-1, keepdim=True) ** 2 / c["channels"] + 1e-6)
        y = y if w is None else y * w
        got = list(torch.autograd.grad(y, [v] if w is None else [v, w], s["dout"].double()))
        if s["dtotal"] is not None:
            got[0] = got[0] + s["dtotal"].double()
        return got
    out, v = [], s["x"].double()
    if s["residual"] is not None:
        v = v + s["residual"].double()
        out = [v]
        v = (s["x"].float() + s["residual"].float()).to(s["x"].dtype).double()  # the norm is of the sum as it is kept
    y = v / torch.sqrt(torch.linalg.vector_norm(v, dim=-1, keepdim=True) ** 2 / c["channels"] + 1e-6)
    y = y if w is None else y * w.double()
    if c["out"] == "same":
        return out + [y]
    top = torch.linalg.vector_norm(y, ord=math.inf, dim=-1)
    scale = torch.where(top == 0, 1.0, top / 448)
    return out + [y / scale[..., None], scale]


def _exact_act(name, v):
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))


def _exact_ffn(s):
    c = s["case"]
    if c["backward"]:
        g, u = s["g"].double().requires_grad_(), s["u"].double().requires_grad_()
        dg, du = torch.autograd.grad(_exact_act(c["act"], g) * u, [g, u], s["dout"].double())
        dx = torch.einsum("mf,fd->md", dg, s["wg"].double()) + torch.einsum("mf,fd->md", du, s["wu"].double())
        out = [dx] + [torch.einsum("mf,md->fd", d, s["x"].double()) for d in (dg, du)]
        return out + [torch.einsum("mf->f", d) for d in (dg, du)] if c["bias"] else out
    x = s["x"].double() if s["xs"] is None else s["x"].double() * s["xs"].double()[:, None]
    pre = []
    for w, scale, b in ((s["wg"], s["gs"], s["bg"]), (s["wu"], s["us"], s["bu"])):
        w = w.double() if scale is None else w.double() * scale.double()[:, None]
        v = torch.einsum("md,fd->mf", x, w)
        pre.append(v if b is None else v + b.double())
    h = _exact_act(c["act"], pre[0]) * pre[1]
    return [h, *pre] if c["saved"] else [h]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "ffn":
        return _exact_ffn(s)
    norm = torch.stack([torch.linalg.vector_norm(v, dtype=torch.float64) for v in (s["matrices"], s["vectors"])]).norm()
    factor = s["limit"] / torch.clamp(norm, min=s["limit"])
    return [norm, s["matrices"].double() * factor, s["vectors"].double() * factor]
