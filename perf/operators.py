"""The rotary-position and group-norm operators, as cases to be measured.

Two operators, each with its gradient:

* rope: q and k of an attention layer turned by positions with several axes
  (time, height, width), with an optional per-head RMS norm of q and k in
  front of the rotation;
* gn: group norm over channels-last pixels with an optional SiLU.

`run` makes the framework's calls where `own` is true and computes the plain
form (elementary torch operations, 32 bits, rounded once) where it is false.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _rope(name, dtype, batch, tokens, q_heads, k_heads, head_dim, axes, style="interleaved", norm=False,
          backward=False, layout="tokens", pos="grid", cond=0, start=0):
    """layout: tokens = [B, N, H, d]; packed = sections of one [B, N, Hq + 2 Hk, d] projection; heads = [B, H, N, d].
    pos: grid = int32 [N, axes] of a token grid; batch = int32 [B, N, axes], another grid per
    batch element; float = float32 [N, axes], a grid stretched to another resolution.
    cond: tokens in front of the grid at position 0 (condition tokens); start: position of the first token."""
    return dict(name=name, op="rope", dtype=dtype, batch=batch, tokens=tokens, q_heads=q_heads, k_heads=k_heads,
                head_dim=head_dim, axes=",".join(map(str, axes)), style=style, norm=norm, backward=backward,
                layout=layout, pos=pos, cond=cond, start=start)


def _gn(name, dtype, batch, pixels, channels, groups, act="silu", affine=True, backward=False, pad=0):
    """pad: channels between one pixel's and the next's (a slice of a wider buffer)."""
    return dict(name=name, op="gn", dtype=dtype, batch=batch, pixels=pixels, channels=channels, groups=groups,
                act=act, affine=affine, backward=backward, pad=pad)


def listed():
    return [
        # one token of a video model's width: nothing but latency
        _rope("rope_norm_one_token", "bf16", 1, 1, 12, 12, 128, (44, 42, 42), norm=True),
        # 81 frames of 480x832 as 32760 tokens, conditional and unconditional pass of one step
        _rope("rope_video_pair", "bf16", 2, 32760, 12, 12, 128, (44, 42, 42)),
        # the same tokens with q/k norm, straight out of the packed projection
        _rope("rope_norm_video", "bf16", 1, 32760, 12, 12, 128, (44, 42, 42), norm=True, layout="packed"),
        # a 1024x1024 image behind 512 condition tokens; shared key heads, head-major, part of each head turned
        _rope("rope_joint_image", "f16", 2, 4608, 16, 4, 128, (0, 48, 48), style="split", layout="heads", cond=512),
        # fine-tuning the video model: gradients of q, k and both norm weights
        _rope("rope_norm_video_grad", "bf16", 1, 32760, 12, 12, 128, (44, 42, 42), norm=True, backward=True),
        # a small odd batch in 32 bits, stretched positions, head width that is no power of two
        _rope("rope_norm_odd_grad", "f32", 3, 1237, 5, 5, 72, (24, 24, 24), style="split", norm=True, backward=True,
              pos="float"),
        # a 16x16 feature map: latency
        _gn("gn_small_map", "bf16", 2, 16 * 16, 512, 32),
        # 21 latent frames of 60x104, each normalised by itself
        _gn("gn_video_frames", "bf16", 21, 60 * 104, 384, 32),
        # 5 frames of 120x208 normalised as one volume
        _gn("gn_volume", "f16", 1, 5 * 120 * 208, 192, 32),
        # the last level of a decoder for a 1024x1024 image
        _gn("gn_decoder_top", "bf16", 1, 1024 * 1024, 128, 32),
        # training an autoencoder's 128x128 level
        _gn("gn_middle_grad", "bf16", 4, 128 * 128, 512, 32, backward=True),
        # 32 bits, odd maps, five channels a group, a slice of a wider buffer
        _gn("gn_odd_grad", "f32", 3, 37 * 53, 60, 12, backward=True, pad=4),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    if rng.random() < 0.5:
        head_dim = rng.choice([32, 64, 72, 80, 96, 128, 128, 128, 160, 256])
        n_axes = rng.choice([1, 2, 3, 3, 4])
        turned = head_dim if rng.random() < 0.7 else head_dim // 2 // 2 * 2
        cuts = sorted(rng.randint(0, turned // 2) for _ in range(n_axes - 1))
        axes = [2 * (b - a) for a, b in zip([0] + cuts, cuts + [turned // 2])]
        q_heads = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 20, 24])
        k_heads = rng.choice([h for h in (1, 2, 3, 4, 5, 8, 12, 16, 20, 24) if q_heads % h == 0])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        norm, backward = rng.random() < 0.5, rng.random() < 0.4
        batch = rng.choice([1, 1, 2, 3, 4])
        row = (q_heads + k_heads) * head_dim * (4 if dtype == "f32" else 2) * 3 * batch
        most = max(1, min(70000, 700_000_000 // row))
        tokens = _log_int(rng, 1, most)
        return {k: v for k, v in _rope("", dtype, batch, tokens, q_heads, k_heads, head_dim, axes,
                                       style=rng.choice(["interleaved", "split"]), norm=norm, backward=backward,
                                       layout=rng.choice(["tokens", "packed", "heads"]),
                                       pos=rng.choice(["grid", "batch", "float"]),
                                       cond=rng.choice([0, 0, tokens // 7]),
                                       start=rng.choice([0, 0, 100_000])).items() if k != "name"}
    groups = rng.choice([1, 2, 4, 8, 16, 32, 32, 32])
    channels = groups * _log_int(rng, 1, min(64, 2048 // groups))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    backward = rng.random() < 0.4
    batch = _log_int(rng, 1, 32)
    least = -(-64 // (channels // groups))  # groups of fewer values leave gradients of nothing but rounding
    most = max(2 * least, min(1 << 20, 250_000_000 // (batch * channels * (4 if dtype == "f32" else 2))))
    pixels = _log_int(rng, least, most)
    return {k: v for k, v in _gn("", dtype, batch, pixels, channels, groups, act=rng.choice(["silu", "silu", "none"]),
                                 affine=rng.random() < 0.85, backward=backward,
                                 pad=rng.choice([0, 0, 0, 8, 5])).items() if k != "name"}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _positions(case, g):
    B, N, cond, start = case["batch"], case["tokens"], case["cond"], case["start"]
    n = len(case["axes"].split(","))
    i = torch.arange(N - cond, device="cuda")
    side = max(1, round((N - cond) ** (1 / max(1, n))))
    at = torch.stack([i // side ** (n - 1 - a) % (side if a else 1 << 30) for a in range(n)], -1) + start
    at = torch.cat([torch.zeros(cond, n, dtype=at.dtype, device="cuda"), at])
    if case["pos"] == "batch":
        shift = torch.randint(0, 64, (B, 1, n), device="cuda", generator=g)
        return (at[None] + shift).to(torch.int32)
    if case["pos"] == "float":
        return at.float() * 0.8125 + torch.rand(n, device="cuda", generator=g)
    return at.to(torch.int32)


def _views(case, g, fill):
    """q and k views of the case's layout; filled with values or left as they are."""
    B, N, Hq, Hk, d = (case[k] for k in ("batch", "tokens", "q_heads", "k_heads", "head_dim"))
    t = _DTYPES[case["dtype"]]

    def new(*shape):
        if not fill:
            return torch.empty(shape, dtype=t, device="cuda")
        return torch.randn(shape, dtype=torch.float32, device="cuda", generator=g).to(t)

    if case["layout"] == "packed" and fill:
        both = new(B, N, Hq + 2 * Hk, d)
        return both[:, :, :Hq], both[:, :, Hq:Hq + Hk]
    if case["layout"] == "heads":
        return new(B, Hq, N, d).transpose(1, 2), new(B, Hk, N, d).transpose(1, 2)
    return new(B, N, Hq, d), new(B, N, Hk, d)


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "rope":
        d = case["head_dim"]
        s["axes"] = tuple(int(a) for a in case["axes"].split(","))
        # which axis turns each pair, and its frequency: a program without the operator keeps these beside its model
        s["axis"] = torch.tensor([a for a, w in enumerate(s["axes"]) for _ in range(w // 2)], device="cuda")
        s["freq"] = torch.tensor([1e4 ** (-2.0 * j / w) for w in s["axes"] for j in range(w // 2)],
                                 dtype=torch.float64, device="cuda")
        s["pos"] = _positions(case, g)
        s["q"], s["k"] = _views(case, g, True)
        s["q_out"], s["k_out"] = _views(case, g, False)
        s["wq"] = s["wk"] = s["dwq"] = s["dwk"] = None
        if case["norm"]:
            s["wq"], s["wk"] = (1 + 0.1 * torch.randn(2, d, device="cuda", generator=g)).unbind()
            s["dwq"], s["dwk"] = torch.empty(2, d, device="cuda").unbind()
        if case["backward"]:
            s["dq_out"], s["dk_out"] = _views(dict(case, layout="tokens"), g, True)
        return s
    B, P, C, G = case["batch"], case["pixels"], case["channels"], case["groups"]
    t = _DTYPES[case["dtype"]]

    def new():
        return torch.empty((B, P, C + case["pad"]), dtype=t, device="cuda")

    s["x"] = new()
    s["x"].copy_(torch.randn(s["x"].shape, device="cuda", generator=g))
    s["x"] = s["x"][..., :C]
    s["x"].mul_((0.5 + torch.rand(C, device="cuda", generator=g)).to(t))
    s["x"].add_(torch.randn(C, device="cuda", generator=g).to(t))
    s["y"] = torch.empty((B, P, C), dtype=t, device="cuda")
    s["mean"], s["rstd"] = torch.empty(2, B, G, device="cuda").unbind()
    s["w"] = s["b"] = s["dw"] = s["db"] = None
    if case["affine"]:
        s["w"] = 1 + 0.2 * torch.randn(C, device="cuda", generator=g)
        s["b"] = 0.3 * torch.randn(C, device="cuda", generator=g)
        s["dw"], s["db"] = torch.empty(2, C, device="cuda").unbind()
    if case["backward"]:
        # what the forward pass left behind
        xg = s["x"].reshape(B, P, G, C // G)
        mean = xg.mean((1, 3), dtype=torch.float64)
        square = torch.linalg.vector_norm(xg, dim=(1, 3), dtype=torch.float64).square() / (P * (C // G))
        s["mean"].copy_(mean)
        s["rstd"].copy_((square - mean.square()).clamp_min(0).add(1e-6).rsqrt())
        s["dy"] = torch.randn((B, P, C), device="cuda", generator=g).to(t)
        s["dx"] = s.pop("y")
    return s


# ------------------------------------------------------------------ plain forms
def _angles(pos, axis, freq):
    """cos and sin [B or 1, N, 1, pairs]: angles in 64 bits, far positions times small frequencies."""
    angle = pos.double()[..., axis] * freq
    angle = angle.reshape(-1, *angle.shape[-2:])[:, :, None]
    return angle.cos().float(), angle.sin().float()


def _turn(x, cos, sin, style):
    half = cos.shape[-1]
    if style == "interleaved":
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def _norm_turn(x, w, cos, sin, style):
    z = x.float()
    if w is not None:
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + 1e-6) * w
    return _turn(z, cos, sin, style).to(x.dtype)


def _norm_turn_grad(x, w, dy, cos, sin, style):
    g = _turn(dy.float(), cos, -sin, style)
    if w is None:
        return g.to(dy.dtype), None
    x = x.float()
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    xhat = x * rstd
    dw = (g * xhat).sum((0, 1, 2))
    g = g * w
    dx = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    return dx.to(dy.dtype), dw


def _plain_rope(s):
    c = s["case"]
    cos, sin = _angles(s["pos"], s["axis"], s["freq"])
    if not c["backward"]:
        return [_norm_turn(s["q"], s["wq"], cos, sin, c["style"]), _norm_turn(s["k"], s["wk"], cos, sin, c["style"])]
    dq, dwq = _norm_turn_grad(s["q"], s["wq"], s["dq_out"], cos, sin, c["style"])
    dk, dwk = _norm_turn_grad(s["k"], s["wk"], s["dk_out"], cos, sin, c["style"])
    return [dq, dk, dwq, dwk] if c["norm"] else [dq, dk]


def _plain_gn(s):
    c, x, w, b = s["case"], s["x"], s["w"], s["b"]
    B, P, C = x.shape
    G = c["groups"]
    v = x.float().reshape(B, P, G, C // G)
    if c["backward"]:
        mean, rstd = s["mean"][:, None, :, None], s["rstd"][:, None, :, None]
    else:
        mean = v.mean((1, 3), keepdim=True)
        rstd = torch.rsqrt((v - mean).square().mean((1, 3), keepdim=True) + 1e-6)
    xhat = (v - mean) * rstd
    z = xhat.reshape(B, P, C)
    if w is not None:
        z = z * w + b
    if not c["backward"]:
        y = z * torch.sigmoid(z) if c["act"] == "silu" else z
        return [y.to(x.dtype), mean.reshape(B, G), rstd.reshape(B, G)]
    dz = s["dy"].float()
    if c["act"] == "silu":
        sig = torch.sigmoid(z)
        dz = dz * (sig * (1 + z * (1 - sig)))
    dw, db = (dz * xhat.reshape(B, P, C)).sum((0, 1)), dz.sum((0, 1))
    g = (dz if w is None else dz * w).reshape(B, P, G, C // G)
    dx = rstd * (g - g.mean((1, 3), keepdim=True) - xhat * (g * xhat).mean((1, 3), keepdim=True))
    dx = dx.reshape(B, P, C).to(x.dtype)
    return [dx] if w is None else [dx, dw, db]


# ------------------------------------------------------------------ the framework's calls
def _own_rope(s):
    from diffusion_transformer_denoising_gb300 import dit

    c = s["case"]
    style = dit.ROPE_INTERLEAVED if c["style"] == "interleaved" else dit.ROPE_SPLIT
    if not c["backward"]:
        dit.dit_rope_forward(s["pos"], s["q"], s["q_out"], s["k"], s["k_out"], axes=s["axes"], theta=1e4, style=style,
                             q_weight=s["wq"], k_weight=s["wk"], eps=1e-6)
        return [s["q_out"], s["k_out"]]
    dit.dit_rope_backward(s["pos"], s["dq_out"], s["q_out"], s["dk_out"], s["k_out"], axes=s["axes"], theta=1e4,
                          style=style, q=s["q"], k=s["k"], q_weight=s["wq"], k_weight=s["wk"],
                          dq_weight=s["dwq"], dk_weight=s["dwk"], eps=1e-6)
    return [s["q_out"], s["k_out"], s["dwq"], s["dwk"]] if c["norm"] else [s["q_out"], s["k_out"]]


def _own_gn(s):
    from diffusion_transformer_denoising_gb300 import dit

    c = s["case"]
    act = dit.ACT_SILU if c["act"] == "silu" else dit.ACT_NONE
    if not c["backward"]:
        dit.dit_group_norm_forward(s["x"], s["y"], c["groups"], weight=s["w"], bias=s["b"], mean=s["mean"],
                                   rstd=s["rstd"], eps=1e-6, act=act)
        return [s["y"], s["mean"], s["rstd"]]
    dit.dit_group_norm_backward(s["x"], s["dy"], s["mean"], s["rstd"], s["dx"], c["groups"], weight=s["w"],
                                bias=s["b"], dweight=s["dw"], dbias=s["db"], act=act)
    return [s["dx"], s["dw"], s["db"]] if c["affine"] else [s["dx"]]


def run(state):
    if own:
        return _own_rope(state) if state["case"]["op"] == "rope" else _own_gn(state)
    return _plain_rope(state) if state["case"]["op"] == "rope" else _plain_gn(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        n = len(case["axes"].split(","))
        rows = case["batch"] * case["tokens"] * (case["q_heads"] + case["k_heads"])
        values = rows * case["head_dim"]
        pos = case["tokens"] * n * 4 * (case["batch"] if case["pos"] == "batch" else 1)
        w = 2 * case["head_dim"] * 4 if case["norm"] else 0
        passes = 3 if case["backward"] and case["norm"] else 2
        each = 3 + (0 if not case["norm"] else 12 if case["backward"] else 4)
        return {"bytes": passes * values * e + pos + w * (2 if case["backward"] else 1), "flops": values * each}
    values = case["batch"] * case["pixels"] * case["channels"]
    stats = case["batch"] * case["groups"] * 8
    w = 8 * case["channels"] if case["affine"] else 0
    passes = 3 if case["backward"] else 2
    each = (16 if case["backward"] else 8) + (8 if case["act"] == "silu" else 0)
    return {"bytes": passes * values * e + stats + w * (2 if case["backward"] else 1), "flops": values * each}


# ------------------------------------------------------------------ 64 bits
def _exact_turn(x, pos, axes, style):
    """The rotation as a product of complex numbers."""
    spins = [pos.double()[..., a:a + 1] * torch.exp(torch.arange(0, w, 2, dtype=torch.float64, device=pos.device)
                                                    * (-math.log(1e4) / w)) for a, w in enumerate(axes) if w]
    spin = torch.cat(spins, -1)
    spin = torch.polar(torch.ones_like(spin), spin).unsqueeze(-2)
    turned, rest = x[..., :2 * spin.shape[-1]], x[..., 2 * spin.shape[-1]:]
    if style == "interleaved":
        v = torch.view_as_complex(turned.unflatten(-1, (-1, 2)).contiguous()) * spin
        out = torch.view_as_real(v).flatten(-2)
    else:
        v = torch.complex(*(h.contiguous() for h in turned.chunk(2, -1))) * spin
        out = torch.cat((v.real, v.imag), -1)
    return torch.cat((out, rest), -1)


def _exact_norm(x, w):
    if w is None:
        return x
    return x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + 1e-6) * w


def exact(case, seed):
    s = prepare(case, seed)
    t = _DTYPES[case["dtype"]]
    grads = []
    if case["op"] == "rope":
        out = []
        for x, w, dy in ((s["q"], s["wq"], s.get("dq_out")), (s["k"], s["wk"], s.get("dk_out"))):
            x = x.double().requires_grad_(case["backward"])
            w = None if w is None else w.double().requires_grad_(case["backward"])
            y = _exact_turn(_exact_norm(x, w), s["pos"], s["axes"], case["style"])
            if not case["backward"]:
                out.append(y)
                continue
            got = torch.autograd.grad(y, [x] if w is None else [x, w], dy.double())
            out.append(got[0])
            grads += got[1:]
        return out + grads
    B, P, C, G = case["batch"], case["pixels"], case["channels"], case["groups"]
    x = s["x"].double().requires_grad_(case["backward"])
    w, b = (None if v is None else v.double().requires_grad_(case["backward"]) for v in (s["w"], s["b"]))
    groups = x.unflatten(-1, (G, C // G)).transpose(1, 2).flatten(2)
    var, mean = torch.var_mean(groups, -1, correction=0)
    rstd = 1 / torch.sqrt(var + 1e-6)
    z = ((groups - mean[..., None]) * rstd[..., None]).unflatten(-1, (P, C // G)).transpose(1, 2).flatten(2)
    if w is not None:
        z = z * w + b
    y = z / (1 + torch.exp(-z)) if case["act"] == "silu" else z
    if not case["backward"]:
        return [y, mean, rstd]
    return list(torch.autograd.grad(y, [x] if w is None else [x, w, b], s["dy"].double()))
