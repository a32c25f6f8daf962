"""ctypes binding of libdit.so: the same entry points as include/dit.h, with
argument marshalling only (every step of the denoiser runs in the library's
CUDA kernels).  Tensors are passed by pointer: torch CUDA tensors (or any
object with data_ptr()) for device buffers, numpy arrays for host buffers.

The library is loaded on first use.  If it has not been built the binding
raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
# DIT_LIB selects another build of the same library (the debug build with
# device-side bounds checks, libdit_debug.so); default: the release build.
LIB_PATH = os.environ.get("DIT_LIB") or os.path.join(_PKG, "libdit.so")

DIT_OK, DIT_ERR_INVALID_ARG, DIT_ERR_SHAPE, DIT_ERR_NOT_LOADED, DIT_ERR_OOM, DIT_ERR_CUDA, DIT_ERR_TIMEOUT = range(7)
PREC_BF16, PREC_F32, PREC_FP8 = 0, 1, 2
COND_CROSS, COND_JOINT = 0, 1
DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2
ROPE_INTERLEAVED, ROPE_SPLIT = 0, 1
ROPE_MAX_AXES, ROPE_MAX_HEAD_DIM = 4, 256
POS_I32, POS_F32 = 0, 1
ACT_NONE, ACT_SILU = 0, 1
LOOP_PARTIAL_SCHEDULE = 1
LOOP_CUDA_GRAPH = 2

# every symbol include/dit.h declares
EXPORTS = ["dit_create", "dit_load_weights", "dit_num_params", "dit_param_info", "dit_timestep_modulation",
           "dit_patch_embed", "dit_block_forward", "dit_final_layer", "cfg_combine", "flow_euler_step",
           "dit_denoise_loop", "dit_synchronize", "dit_device_bytes", "dit_destroy", "dit_status_string",
           "dit_last_error", "dit_debug_fail_alloc_after", "dit_debug_gemm_cta_pairs", "dit_debug_stall", "dit_profile_start", "dit_profile_stop",
           "dit_timestep_modulation_noalloc", "dit_rope_forward", "dit_rope_backward", "dit_rope_workspace_bytes",
           "dit_group_norm_forward", "dit_group_norm_backward", "dit_group_norm_workspace_bytes"]
NOALLOC_MAX_BATCH, NOALLOC_MAX_HIDDEN = 64, 262144

KERNEL_KINDS = ["gemm_qkv", "gemm_out", "gemm_cross_q", "gemm_cross_kv", "gemm_ffn1", "gemm_ffn2", "gemm_embed",
                "attn_self", "attn_cross", "ln", "small", "cfg_euler"]


class DitConfig(C.Structure):
    _fields_ = [("in_channels", C.c_int32), ("patch", C.c_int32 * 3), ("hidden", C.c_int32),
                ("heads", C.c_int32), ("head_dim", C.c_int32), ("mlp", C.c_int32), ("depth", C.c_int32),
                ("cond_dim", C.c_int32), ("freq_dim", C.c_int32), ("rope_axes", C.c_int32 * 3),
                ("cond_mode", C.c_int32), ("precision", C.c_int32), ("ln_eps", C.c_float),
                ("rope_theta", C.c_float), ("timestep_scale", C.c_float)]


class DitTensor(C.Structure):
    _fields_ = [("name", C.c_char_p), ("ndim", C.c_int32), ("shape", C.c_int64 * 4), ("dtype", C.c_int32),
                ("data", C.c_void_p)]


class DitError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"[{status}] {msg}")
        self.status = status


_lib = None


def lib():
    """The loaded library (raises if libdit.so has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it first (python -m "
                           "diffusion_transformer_denoising_gb300.build or __graft_entry__.build())")
    L = C.CDLL(LIB_PATH)
    vp, i32, i64, f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_float
    sig = {
        "dit_create": ([C.POINTER(DitConfig), C.c_int, C.POINTER(vp)], C.c_int),
        "dit_load_weights": ([vp, C.POINTER(DitTensor), C.c_int], C.c_int),
        "dit_num_params": ([C.POINTER(DitConfig)], C.c_int),
        "dit_param_info": ([C.POINTER(DitConfig), C.c_int, C.c_char_p, C.c_int, C.POINTER(i32),
                            C.POINTER(i64)], C.c_int),
        "dit_timestep_modulation": ([vp, C.POINTER(f32), C.c_int, vp, vp], C.c_int),
        "dit_timestep_modulation_noalloc": ([vp, C.POINTER(f32), C.c_int, vp, vp], C.c_int),
        "dit_patch_embed": ([vp, vp, C.c_int, C.POINTER(i32), vp, vp], C.c_int),
        "dit_block_forward": ([vp, C.c_int, vp, vp, vp, vp, C.c_int, C.POINTER(i32), C.c_int, vp], C.c_int),
        "dit_final_layer": ([vp, vp, vp, C.c_int, C.POINTER(i32), vp, vp], C.c_int),
        "cfg_combine": ([vp, vp, f32, vp, i64, vp], C.c_int),
        "flow_euler_step": ([vp, vp, f32, f32, i64, vp], C.c_int),
        "dit_denoise_loop": ([vp, vp, C.c_int, C.POINTER(i32), vp, vp, C.c_int, C.POINTER(f32), C.c_int, f32,
                              C.c_uint32, vp], C.c_int),
        "dit_synchronize": ([vp, vp], C.c_int),
        "dit_device_bytes": ([vp], i64),
        "dit_destroy": ([vp], None),
        "dit_status_string": ([C.c_int], C.c_char_p),
        "dit_last_error": ([], C.c_char_p),
        "dit_debug_fail_alloc_after": ([C.c_int], None),
        "dit_debug_gemm_cta_pairs": ([C.c_int], None),
        "dit_debug_stall": ([vp, vp], C.c_int),
        "dit_profile_start": ([vp, C.c_int], C.c_int),
        "dit_profile_stop": ([vp, C.POINTER(i64), C.POINTER(C.c_double)], C.c_int),
        "dit_rope_forward": ([vp, vp], C.c_int),
        "dit_rope_backward": ([vp, vp, i64, vp], C.c_int),
        "dit_rope_workspace_bytes": ([vp], i64),
        "dit_group_norm_forward": ([vp, vp, i64, vp], C.c_int),
        "dit_group_norm_backward": ([vp, vp, i64, vp], C.c_int),
        "dit_group_norm_workspace_bytes": ([vp, C.c_int], i64),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def _check(status: int):
    if status != DIT_OK:
        raise DitError(status, lib().dit_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if hasattr(t, "data_ptr"):
        return C.c_void_p(t.data_ptr())
    if isinstance(t, np.ndarray):
        return C.c_void_p(t.ctypes.data)
    if isinstance(t, int):
        return C.c_void_p(t)
    raise TypeError(f"cannot take a pointer of {type(t)}")


def _stream(stream):
    if stream is None:
        try:
            import torch
            if torch.cuda.is_available():
                return C.c_void_p(torch.cuda.current_stream().cuda_stream)
        except Exception:
            pass
        return None
    if hasattr(stream, "cuda_stream"):
        return C.c_void_p(stream.cuda_stream)
    return C.c_void_p(int(stream))


def make_config(cfg: dict) -> DitConfig:
    c = DitConfig()
    c.in_channels = cfg["in_channels"]
    c.patch[:] = list(cfg["patch"])
    for k in ("hidden", "heads", "head_dim", "mlp", "depth", "cond_dim", "freq_dim", "cond_mode", "precision"):
        setattr(c, k, int(cfg[k]))
    c.rope_axes[:] = list(cfg["rope_axes"])
    c.ln_eps, c.rope_theta, c.timestep_scale = cfg["ln_eps"], cfg["rope_theta"], cfg["timestep_scale"]
    return c


def dit_num_params(cfg: dict) -> int:
    return lib().dit_num_params(C.byref(make_config(cfg)))


def dit_param_info(cfg: dict, i: int):
    buf = C.create_string_buffer(256)
    nd = C.c_int32()
    shape = (C.c_int64 * 4)()
    _check(lib().dit_param_info(C.byref(make_config(cfg)), i, buf, 256, C.byref(nd), shape))
    return buf.value.decode(), tuple(shape[: nd.value])


def cfg_combine(vc, vu, g: float, v, n: int, stream=None):
    _check(lib().cfg_combine(_ptr(vc), _ptr(vu), g, _ptr(v), n, _stream(stream)))


def flow_euler_step(x, v, sigma: float, sigma_next: float, n: int, stream=None):
    _check(lib().flow_euler_step(_ptr(x), _ptr(v), sigma, sigma_next, n, _stream(stream)))


# ------------------------------------------------------------- operators
# dit_rope_args and dit_group_norm_args of include/dit.h, packed in one go
_ROPE_ARGS = struct.Struct("<2q8i2fQ2q2i" + 2 * "2iQ3qQ3qQ3q2Q")
_GN_ARGS = struct.Struct("<2q4ifiQ2qQ2qQ2q6Q")
_NO_VIEW = (0, 0, 0, 0)
_dtype_codes = None


def _dtype_code(t):
    global _dtype_codes
    if _dtype_codes is None:
        import torch
        _dtype_codes = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
    try:
        return _dtype_codes[t.dtype]
    except KeyError:
        raise DitError(DIT_ERR_INVALID_ARG, f"unsupported dtype {t.dtype}") from None


def _refuse(status, msg):
    raise DitError(status, msg)


def _param(name, t, shape, device):
    """Pointer of an optional contiguous float32 tensor of this shape."""
    if t is None:
        return 0
    if t.device != device:
        _refuse(DIT_ERR_INVALID_ARG, f"{name} is on {t.device}, not {device}")
    if t.element_size() != 4 or not t.is_floating_point():
        _refuse(DIT_ERR_INVALID_ARG, f"{name} must be float32")
    if tuple(t.shape) != shape or not t.is_contiguous():
        _refuse(DIT_ERR_SHAPE, f"{name} must be contiguous {list(shape)}")
    return t.data_ptr()


def _launch_on(device, workspace, stream, need, args):
    """(workspace pointer, bytes, stream) of a call on `device`."""
    import torch
    if device.type != "cuda":
        _refuse(DIT_ERR_INVALID_ARG, f"tensors are on {device}, not on a CUDA device")
    s = torch.cuda.current_stream(device).cuda_stream if stream is None else _stream(stream)
    if need is None:
        return 0, 0, s
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            _refuse(DIT_ERR_INVALID_ARG, f"the workspace must be contiguous memory on {device}")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), s
    n = need(args)
    if n < 0:
        raise DitError(DIT_ERR_INVALID_ARG, lib().dit_last_error().decode())
    if n == 0:
        return 0, 0, s
    if stream is not None:
        _refuse(DIT_ERR_INVALID_ARG, "a call on an explicit stream needs its workspace passed in")
    # torch's allocator hands the block out in the order of the current stream, which is the call's
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    return ws.data_ptr(), n, s


def _heads_view(name, t, like):
    """(pointer, batch, token and head strides) of a [batch, tokens, heads, head_dim] view."""
    if t.shape != like.shape:
        _refuse(DIT_ERR_SHAPE, f"{name} is {list(t.shape)}, not {list(like.shape)}")
    if t.dtype != like.dtype or t.device != like.device:
        _refuse(DIT_ERR_INVALID_ARG, f"{name} has another dtype or device")
    sb, st, sh, sd = t.stride()
    if sd != 1 and t.shape[3] > 1 and t.numel():
        _refuse(DIT_ERR_SHAPE, f"{name}: the channels of a head must be contiguous")
    return t.data_ptr(), sb, st, sh


def _rope_heads(tag, x, dy, out, weight, dweight, ref):
    """Packed dit_rope_heads of one tensor; ref is (batch, tokens, head_dim, dtype, device)."""
    if out is None:
        if x is not None or dy is not None or weight is not None or dweight is not None:
            _refuse(DIT_ERR_INVALID_ARG, f"{tag} is given without its output")
        return (0, 0, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, 0, 0)
    if out.dim() != 4 or (out.shape[0], out.shape[1], out.shape[3]) != ref[:3]:
        _refuse(DIT_ERR_SHAPE, f"{tag} is {list(out.shape)}: [{ref[0]}, {ref[1]}, heads, {ref[2]}] is wanted")
    if out.dtype != ref[3] or out.device != ref[4]:
        _refuse(DIT_ERR_INVALID_ARG, f"{tag} has another dtype or device")
    return (out.shape[2], 0,
            *(_NO_VIEW if x is None else _heads_view(f"{tag} input", x, out)),
            *(_NO_VIEW if dy is None else _heads_view(f"{tag} gradient", dy, out)),
            *_heads_view(f"{tag} output", out, out),
            _param(f"{tag}_weight", weight, (ref[2],), ref[4]), _param(f"d{tag}_weight", dweight, (ref[2],), ref[4]))


def _rope_args(pos, axes, theta, style, eps, first, q, k):
    import torch
    B, N, _, d = first.shape if first.dim() == 4 else _refuse(DIT_ERR_SHAPE, "q must be [batch, tokens, heads, head_dim]")
    n = len(axes)
    if not 1 <= n <= ROPE_MAX_AXES:
        _refuse(DIT_ERR_INVALID_ARG, f"1 to {ROPE_MAX_AXES} axes are supported")
    if pos.dim() not in (2, 3) or tuple(pos.shape[-2:]) != (N, n) or (pos.dim() == 3 and pos.shape[0] != B):
        _refuse(DIT_ERR_SHAPE, f"positions are {list(pos.shape)}: [{N}, {n}] or [{B}, {N}, {n}] is wanted")
    if pos.dtype not in (torch.int32, torch.float32) or pos.device != first.device:
        _refuse(DIT_ERR_INVALID_ARG, "positions must be int32 or float32 on the tensors' device")
    ps = pos.stride()
    if n > 1 and ps[-1] != 1 and pos.numel():
        _refuse(DIT_ERR_SHAPE, "the axes of a position must be contiguous")
    ref = (B, N, d, first.dtype, first.device)
    return _ROPE_ARGS.pack(B, N, d, _dtype_code(first), style, n, *axes, *(0,) * (4 - n), theta, eps, pos.data_ptr(),
                           ps[0] if pos.dim() == 3 else 0, ps[-2], POS_F32 if pos.is_floating_point() else POS_I32, 0,
                           *_rope_heads("q", *q, ref), *_rope_heads("k", *k, ref))


def dit_rope_forward(pos, q, q_out, k=None, k_out=None, *, axes, theta=1e4, style=ROPE_INTERLEAVED, q_weight=None,
                     k_weight=None, eps=1e-6, stream=None):
    """Turn q (and k) [batch, tokens, heads, head_dim] by positions with
    several axes, behind a per-head RMS norm where a weight is given.

    pos: int32 or float32 [tokens, len(axes)], or [batch, tokens, len(axes)];
    axes: rotary channels per axis; q_out / k_out may be q / k themselves.
    Views may have any strides with contiguous heads; k may have its own
    number of heads (see dit_rope_forward in include/dit.h)."""
    args = _rope_args(pos, axes, theta, style, eps, q, (q, None, q_out, q_weight, None),
                      (k, None, k_out, k_weight, None))
    _check(lib().dit_rope_forward(args, _launch_on(q.device, None, stream, None, args)[2]))


def dit_rope_backward(pos, dq_out, dq, dk_out=None, dk=None, *, axes, theta=1e4, style=ROPE_INTERLEAVED, q=None,
                      k=None, q_weight=None, k_weight=None, dq_weight=None, dk_weight=None, eps=1e-6, workspace=None,
                      stream=None):
    """Gradient of dit_rope_forward: dq (and dk) from dq_out (and dk_out);
    with a weight the forward's input q (k) is read, and d{q,k}_weight
    (float32 [head_dim], overwritten) is computed where given.  workspace: a
    contiguous tensor of dit_rope_workspace_bytes, or None to take one from
    torch's allocator (only on torch's current stream)."""
    args = _rope_args(pos, axes, theta, style, eps, dq_out, (q, dq_out, dq, q_weight, dq_weight),
                      (k, dk_out, dk, k_weight, dk_weight))
    L = lib()
    ws, n, s = _launch_on(dq_out.device, workspace, stream,
                          None if dq_weight is None and dk_weight is None else L.dit_rope_workspace_bytes, args)
    _check(L.dit_rope_backward(args, ws, n, s))


def dit_rope_workspace_bytes(head_dim: int) -> int:
    """Workspace of dit_rope_backward when weight gradients are wanted."""
    heads = (1, 0, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, 16, 32)
    none = (0, 0, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, 0, 0)
    n = lib().dit_rope_workspace_bytes(_ROPE_ARGS.pack(1, 1, head_dim, DTYPE_F32, 0, 1, 0, 0, 0, 0, 1e4, 0.0, 0, 0, 0,
                                                       POS_I32, 0, *heads, *none))
    if n < 0:
        raise DitError(DIT_ERR_SHAPE, lib().dit_last_error().decode())
    return n


def _pixel_view(name, t, like):
    """(pointer, batch stride, pixel stride) of a [batch, ..., channels] view."""
    if t.shape != like.shape:
        _refuse(DIT_ERR_SHAPE, f"{name} is {list(t.shape)}, not {list(like.shape)}")
    if t.dtype != like.dtype or t.device != like.device:
        _refuse(DIT_ERR_INVALID_ARG, f"{name} has another dtype or device")
    shape, stride = t.shape, t.stride()
    if t.numel() == 0:
        return 0, 0, 0
    if stride[-1] != 1 and shape[-1] > 1:
        _refuse(DIT_ERR_SHAPE, f"{name}: channels must be contiguous (channels last)")
    step, span = 0, 0
    for i in range(t.dim() - 2, 0, -1):  # the middle axes as one axis of pixels
        if shape[i] == 1:
            continue
        if not step:
            step = stride[i]
        elif stride[i] != span:
            _refuse(DIT_ERR_SHAPE, f"{name}: the axes between batch and channels must have one common stride")
        span = stride[i] * shape[i]
    return t.data_ptr(), stride[0] if shape[0] > 1 else 0, step


def _gn_args(x, dy, out, groups, weight, bias, mean, rstd, dweight, dbias, eps, act):
    if x.dim() < 3:
        _refuse(DIT_ERR_SHAPE, "x must be [batch, ..., channels]")
    B, C = x.shape[0], x.shape[-1]
    P = 1
    for v in x.shape[1:-1]:
        P *= v
    dev = x.device
    return _GN_ARGS.pack(B, P, C, groups, _dtype_code(x), act, eps, 0, *_pixel_view("x", x, x),
                         *((0, 0, 0) if dy is None else _pixel_view("dy", dy, x)), *_pixel_view("out", out, x),
                         _param("weight", weight, (C,), dev), _param("bias", bias, (C,), dev),
                         _param("mean", mean, (B, groups), dev), _param("rstd", rstd, (B, groups), dev),
                         _param("dweight", dweight, (C,), dev), _param("dbias", dbias, (C,), dev))


def dit_group_norm_forward(x, y, groups: int, *, weight=None, bias=None, mean=None, rstd=None, eps=1e-6, act=ACT_NONE,
                           workspace=None, stream=None):
    """Group norm of x [batch, ..., channels] (channels last) with an
    activation, into y (which may be x).  mean / rstd: float32 [batch, groups]
    written for the backward call, or None.  workspace: a contiguous tensor of
    dit_group_norm_workspace_bytes, or None to take one from torch's allocator
    (only on torch's current stream)."""
    args = _gn_args(x, None, y, groups, weight, bias, mean, rstd, None, None, eps, act)
    L = lib()
    ws, n, s = _launch_on(x.device, workspace, stream, lambda a: L.dit_group_norm_workspace_bytes(a, 0), args)
    _check(L.dit_group_norm_forward(args, ws, n, s))


def dit_group_norm_backward(x, dy, mean, rstd, dx, groups: int, *, weight=None, bias=None, dweight=None, dbias=None,
                            act=ACT_NONE, workspace=None, stream=None):
    """Gradient of dit_group_norm_forward: dx (which may be dy or x), and
    dweight / dbias (float32 [channels], overwritten) where given.  mean and
    rstd are what the forward call wrote."""
    args = _gn_args(x, dy, dx, groups, weight, bias, mean, rstd, dweight, dbias, 0.0, act)
    L = lib()
    ws, n, s = _launch_on(x.device, workspace, stream, lambda a: L.dit_group_norm_workspace_bytes(a, 1), args)
    _check(L.dit_group_norm_backward(args, ws, n, s))


def dit_group_norm_workspace_bytes(x, groups: int, backward: bool) -> int:
    """Workspace of a group-norm call on tensors like x (the same strides and
    alignment in every argument)."""
    view = _pixel_view("x", x, x)
    P = 1
    for v in x.shape[1:-1]:
        P *= v
    n = lib().dit_group_norm_workspace_bytes(
        _GN_ARGS.pack(x.shape[0], P, x.shape[-1], groups, _dtype_code(x), ACT_NONE, 0.0, 0, *view, *view, *view,
                      0, 0, 0, 0, 0, 0), 1 if backward else 0)
    if n < 0:
        raise DitError(DIT_ERR_SHAPE, lib().dit_last_error().decode())
    return n


def dit_debug_fail_alloc_after(n: int):
    lib().dit_debug_fail_alloc_after(n)


def dit_debug_gemm_cta_pairs(mode: int):
    """0: GEMMs never on CTA pairs, 1 (default): when the main loop has >= 16
    K blocks, 2: always (widths that are multiples of 256)."""
    lib().dit_debug_gemm_cta_pairs(int(mode))


class DiT:
    """One dit_model: create, load weights, run pieces or the whole loop."""

    def __init__(self, cfg: dict, device: int = 0):
        self.cfg = dict(cfg)
        self._cfg = make_config(cfg)
        h = C.c_void_p()
        _check(lib().dit_create(C.byref(self._cfg), device, C.byref(h)))
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            lib().dit_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def device_bytes(self) -> int:
        return lib().dit_device_bytes(self.h)

    def load_weights(self, weights: dict, chunk: int = 64):
        """weights: name -> numpy float32 array, or torch tensor (float32 or
        bfloat16, host or device)."""
        keep, items = [], list(weights.items())
        for s in range(0, len(items), chunk):
            arr = (DitTensor * len(items[s:s + chunk]))()
            for j, (name, w) in enumerate(items[s:s + chunk]):
                t = arr[j]
                t.name = name.encode()
                keep.append(t.name)
                if isinstance(w, np.ndarray):
                    w = np.ascontiguousarray(w, dtype=np.float32)
                    keep.append(w)
                    t.dtype = DTYPE_F32
                else:
                    import torch
                    w = w.contiguous()
                    keep.append(w)
                    if w.dtype == torch.bfloat16:
                        t.dtype = DTYPE_BF16
                    elif w.dtype == torch.float32:
                        t.dtype = DTYPE_F32
                    else:
                        raise TypeError(f"{name}: unsupported dtype {w.dtype}")
                t.ndim = len(w.shape)
                for d in range(4):
                    t.shape[d] = w.shape[d] if d < len(w.shape) else 1
                t.data = _ptr(w).value
            _check(lib().dit_load_weights(self.h, arr, len(arr)))

    def dit_timestep_modulation(self, t_host, mod, stream=None):
        t = np.ascontiguousarray(t_host, dtype=np.float32)
        _check(lib().dit_timestep_modulation(self.h, t.ctypes.data_as(C.POINTER(C.c_float)), len(t), _ptr(mod),
                                             _stream(stream)))

    def dit_timestep_modulation_noalloc(self, t_host, mod, stream=None):
        """dit_timestep_modulation without any device allocation (fixed
        library scratch; see include/dit.h for the limits)."""
        t = np.ascontiguousarray(t_host, dtype=np.float32)
        _check(lib().dit_timestep_modulation_noalloc(self.h, t.ctypes.data_as(C.POINTER(C.c_float)), len(t),
                                                     _ptr(mod), _stream(stream)))

    def dit_patch_embed(self, latents, batch: int, thw, x, stream=None):
        a = (C.c_int32 * 3)(*thw)
        _check(lib().dit_patch_embed(self.h, _ptr(latents), batch, a, _ptr(x), _stream(stream)))

    def dit_block_forward(self, block: int, x, xc, mod, cond, batch: int, grid, cond_len: int, stream=None):
        g = (C.c_int32 * 3)(*grid)
        _check(lib().dit_block_forward(self.h, block, _ptr(x), _ptr(xc), _ptr(mod), _ptr(cond), batch, g,
                                       cond_len, _stream(stream)))

    def dit_final_layer(self, x, mod, batch: int, thw, v, stream=None):
        a = (C.c_int32 * 3)(*thw)
        _check(lib().dit_final_layer(self.h, _ptr(x), _ptr(mod), batch, a, _ptr(v), _stream(stream)))

    def dit_denoise_loop(self, latents, batch: int, thw, cond, uncond, cond_len: int, sigmas, guidance: float,
                         flags: int = 0, stream=None):
        a = (C.c_int32 * 3)(*thw)
        sg = np.ascontiguousarray(sigmas, dtype=np.float32)
        _check(lib().dit_denoise_loop(self.h, _ptr(latents), batch, a, _ptr(cond), _ptr(uncond), cond_len,
                                      sg.ctypes.data_as(C.POINTER(C.c_float)), len(sg) - 1, guidance, flags,
                                      _stream(stream)))

    def dit_profile_start(self, timing: bool = True):
        _check(lib().dit_profile_start(self.h, 1 if timing else 0))

    def dit_profile_stop(self):
        """{kind: (launches, total device ms)} since dit_profile_start."""
        n = len(KERNEL_KINDS)
        counts, ms = (C.c_int64 * n)(), (C.c_double * n)()
        _check(lib().dit_profile_stop(self.h, counts, ms))
        return {k: (counts[i], ms[i]) for i, k in enumerate(KERNEL_KINDS)}

    def dit_synchronize(self, stream=None):
        _check(lib().dit_synchronize(self.h, _stream(stream)))

    def dit_debug_stall(self, stream=None):
        """Test hook: a device wait that runs out (see include/dit.h)."""
        _check(lib().dit_debug_stall(self.h, _stream(stream)))
