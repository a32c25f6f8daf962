"""ctypes binding of libdit.so: the same entry points as include/dit.h, with
argument marshalling only (every step of the denoiser runs in the library's
CUDA kernels).  Tensors are passed by pointer: torch CUDA tensors (or any
object with data_ptr()) for device buffers, numpy arrays for host buffers.

The library is loaded on first use.  If it has not been built the binding
raises instead of falling back to anything else.
"""
from __future__ import annotations

import array
import ctypes as C
import operator
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
DTYPE_F32, DTYPE_BF16, DTYPE_F16, DTYPE_E4M3 = 0, 1, 2, 3
ROPE_INTERLEAVED, ROPE_SPLIT = 0, 1
ROPE_MAX_AXES, ROPE_MAX_HEAD_DIM = 4, 256
POS_I32, POS_F32 = 0, 1
ACT_NONE, ACT_SILU, ACT_GELU = 0, 1, 2
RMS_NORM_MAX_CHANNELS = 16384
LOOP_PARTIAL_SCHEDULE = 1
LOOP_CUDA_GRAPH = 2

# every symbol include/dit.h declares
EXPORTS = ["dit_create", "dit_load_weights", "dit_num_params", "dit_param_info", "dit_timestep_modulation",
           "dit_patch_embed", "dit_block_forward", "dit_final_layer", "cfg_combine", "flow_euler_step",
           "dit_denoise_loop", "dit_synchronize", "dit_device_bytes", "dit_destroy", "dit_status_string",
           "dit_last_error", "dit_debug_fail_alloc_after", "dit_debug_gemm_cta_pairs", "dit_debug_stall", "dit_profile_start", "dit_profile_stop",
           "dit_timestep_modulation_noalloc", "dit_rope_forward", "dit_rope_backward", "dit_rope_workspace_bytes",
           "dit_group_norm_forward", "dit_group_norm_backward", "dit_group_norm_workspace_bytes",
           "dit_rms_norm_forward", "dit_rms_norm_backward", "dit_rms_norm_workspace_bytes",
           "dit_gated_ffn_forward", "dit_gated_ffn_backward", "dit_gated_ffn_workspace_bytes",
           "dit_gated_ffn_synchronize", "dit_grad_norm", "dit_grad_norm_workspace_bytes"]
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
        "dit_rms_norm_forward": ([vp, vp], C.c_int),
        "dit_rms_norm_backward": ([vp, vp, i64, vp], C.c_int),
        "dit_rms_norm_workspace_bytes": ([vp], i64),
        "dit_gated_ffn_forward": ([vp, vp, i64, vp], C.c_int),
        "dit_gated_ffn_backward": ([vp, vp, i64, vp], C.c_int),
        "dit_gated_ffn_workspace_bytes": ([vp, C.c_int], i64),
        "dit_gated_ffn_synchronize": ([vp], C.c_int),
        "dit_grad_norm": ([vp, i64, f32, vp, vp, i64, vp], C.c_int),
        "dit_grad_norm_workspace_bytes": ([vp, i64], i64),
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
# the argument structures of include/dit.h, packed in one go
_ROPE_ARGS = struct.Struct("<2q8i2fQ2q2i" + 2 * "2iQ3qQ3qQ3q2Q")
_GN_ARGS = struct.Struct("<2q4ifiQ2qQ2qQ2q6Q")
_NORM_ARGS = struct.Struct("<2q3if" + 5 * "Q2q" + "3Q")
_FFN_ARGS = struct.Struct("<q6i" + 3 * "Qq" + "5Q" + 6 * "Qq" + "2Q")
_INF = float("inf")
_NO_VIEW = (0, 0, 0, 0)
_torch = None          # the module, its dtypes as dit.h names them and its grad mode, on first use
_dtype_codes = {}
_operand_codes = {}    # and e4m3
_grad_mode = None
_forward_ad = None


def _use_torch():
    global _torch, _grad_mode, _forward_ad
    if _torch is None:
        import torch
        import torch.autograd.forward_ad
        _grad_mode, _forward_ad = torch.is_grad_enabled, torch.autograd.forward_ad
        _dtype_codes.update({torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16})
        _operand_codes.update(_dtype_codes)
        _operand_codes[torch.float8_e4m3fn] = DTYPE_E4M3
        _torch = torch
    return _torch


def _refuse(status, msg):
    raise DitError(status, msg)


def _refuse_scalar(e):
    raise DitError(DIT_ERR_INVALID_ARG, f"an argument has the wrong type or does not fit its field: {e}") from None


def _dtype_code(dtype):
    code = _dtype_codes.get(dtype)
    return _refuse(DIT_ERR_INVALID_ARG, f"unsupported dtype {dtype}") if code is None else code


# The library looks up which device owns each pointer and refuses a mixture,
# so the helpers here compare types and shapes only.
def _param(name, t, shape):
    """Pointer of an optional contiguous float32 tensor of this shape."""
    if t is None:
        return 0
    if t.dtype is not _torch.float32:
        _refuse(DIT_ERR_INVALID_ARG, f"{name}: weights and statistics must be float32")
    if t.shape != shape or not t.is_contiguous():
        _refuse(DIT_ERR_SHAPE, f"{name}: weights and statistics must be contiguous, here {list(shape)}")
    return t.data_ptr()


def _refuse_autograd():
    """The calls write into the tensors they are given and record nothing, so inputs that autograd waits for a gradient
    of are refused."""
    _refuse(DIT_ERR_INVALID_ARG, "a tensor requires grad: autograd does not see this call (run it under torch.no_grad(), "
                                 "or inside a torch.autograd.Function with the backward call)")


def _refuse_tangents(*inputs):
    """Inside a dual level of torch.autograd.forward_ad (whatever the grad mode is): inputs with a tangent are refused, for
    the calls write values only."""
    for t in inputs:
        if t is not None and _forward_ad.unpack_dual(t).tangent is not None:
            _refuse(DIT_ERR_INVALID_ARG, "a tensor has a forward-mode tangent, which this call would lose (unpack the dual tensor)")


def _raw_stream(t, stream):
    """cudaStream_t of the call: torch's current stream of the tensor's device unless one is given."""
    if not t.is_cuda:
        _refuse(DIT_ERR_INVALID_ARG, f"tensors are on {t.device}, not on a CUDA device")
    return _torch._C._cuda_getCurrentRawStream(t.device.index) if stream is None else _stream(stream)


def _workspace(t, workspace, stream, need):
    """(pointer, bytes, owner) of the caller's workspace, or of one taken from
    torch's allocator: its owner lives until the launch has been made."""
    if workspace is not None:
        if not workspace.is_contiguous():
            _refuse(DIT_ERR_INVALID_ARG, "the workspace must be contiguous")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if need < 0:
        raise DitError(DIT_ERR_INVALID_ARG, lib().dit_last_error().decode())
    if need == 0:
        return 0, 0, None
    if stream is not None:
        _refuse(DIT_ERR_INVALID_ARG, "a call on an explicit stream needs its workspace passed in")
    # the allocator hands blocks out in the order of the current stream, which is the call's
    ws = _torch.empty(need, dtype=_torch.uint8, device=t.device)
    return ws.data_ptr(), need, ws


def _bad_view(tag, t, shape, dtype):
    if t.shape != shape:
        _refuse(DIT_ERR_SHAPE, f"{tag} tensor is {list(t.shape)}, not {list(shape)}")
    if t.dtype is not dtype:
        _refuse(DIT_ERR_INVALID_ARG, f"{tag} tensor is {t.dtype}, not {dtype}")
    _refuse(DIT_ERR_SHAPE, f"{tag}: the channels of a head must be contiguous")


def _heads_view(tag, t, shape, dtype):
    """(pointer, batch, token and head strides) of a [batch, tokens, heads, head_dim] view."""
    if t is None:
        return _NO_VIEW
    sb, st, sh, sd = t.stride() if t.dim() == 4 else _NO_VIEW
    if t.shape != shape or t.dtype is not dtype or (sd != 1 and t.numel()):
        _bad_view(tag, t, shape, dtype)
    return t.data_ptr(), sb, st, sh


_NO_HEADS = (0, 0, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, 0, 0)


def _rope_heads(tag, x, dy, out, weight, dweight, B, N, d, dtype):
    """Fields of the dit_rope_heads of one tensor."""
    if out is None:
        if x is not None or dy is not None or weight is not None or dweight is not None:
            _refuse(DIT_ERR_INVALID_ARG, f"{tag} is given without its output")
        return _NO_HEADS
    shape = out.shape
    if len(shape) != 4 or shape[0] != B or shape[1] != N or shape[3] != d:
        _refuse(DIT_ERR_SHAPE, f"{tag} output is {list(shape)}: [{B}, {N}, heads, {d}] is wanted")
    return (shape[2], 0, *_heads_view(tag, x, shape, dtype), *_heads_view(tag, dy, shape, dtype),
            *_heads_view(tag, out, shape, dtype), 0 if weight is None else _param(tag, weight, (d,)),
            0 if dweight is None else _param(tag, dweight, (d,)))


def _rope_args(pos, axes, theta, style, eps, first, q, k):
    torch = _torch or _use_torch()
    if _grad_mode():
        if pos.requires_grad:
            _refuse_autograd()
        for x, dy, _, weight, _ in (q, k):
            if (x is not None and x.requires_grad or weight is not None and weight.requires_grad or
                    dy is not None and dy.requires_grad):
                _refuse_autograd()
    if _forward_ad._current_level >= 0:
        _refuse_tangents(pos, *q[:2], q[3], *k[:2], k[3])
    if first.dim() != 4:
        _refuse(DIT_ERR_SHAPE, "q must be [batch, tokens, heads, head_dim]")
    B, N, _, d = first.shape
    dtype, n, ps, pd = first.dtype, len(axes), pos.shape, pos.dtype
    code = _dtype_code(dtype)
    if not 1 <= n <= ROPE_MAX_AXES:
        _refuse(DIT_ERR_INVALID_ARG, f"1 to {ROPE_MAX_AXES} axes are supported")
    if len(ps) not in (2, 3) or ps[-2] != N or ps[-1] != n or (len(ps) == 3 and ps[0] != B):
        _refuse(DIT_ERR_SHAPE, f"positions are {list(ps)}: [{N}, {n}] or [{B}, {N}, {n}] is wanted")
    if pd is not torch.int32 and pd is not torch.float32:
        _refuse(DIT_ERR_INVALID_ARG, "positions must be int32 or float32")
    st = pos.stride()
    if st[-1] != 1 and n > 1 and pos.numel():
        _refuse(DIT_ERR_SHAPE, "the axes of a position must be contiguous")
    try:
        return _ROPE_ARGS.pack(B, N, d, code, style, n, *axes, *_NO_VIEW[n:], theta, eps, pos.data_ptr(),
                               st[0] if len(ps) == 3 else 0, st[-2], POS_I32 if pd is torch.int32 else POS_F32, 0,
                               *_rope_heads("q", *q, B, N, d, dtype), *_rope_heads("k", *k, B, N, d, dtype))
    except (struct.error, OverflowError) as e:
        _refuse_scalar(e)


def dit_rope_forward(pos, q, q_out, k=None, k_out=None, *, axes, theta=1e4, style=ROPE_INTERLEAVED, q_weight=None,
                     k_weight=None, eps=1e-6, stream=None):
    """Turn q (and k) [batch, tokens, heads, head_dim] by positions with
    several axes, behind a per-head RMS norm where a weight is given.

    pos: int32 or float32 [tokens, len(axes)], or [batch, tokens, len(axes)];
    axes: rotary channels per axis; q_out / k_out may be q / k themselves.
    Views may have any strides with contiguous heads; k may have its own
    number of heads (see dit_rope_forward in include/dit.h).  Nothing is
    recorded for autograd, so with grad mode on an input that requires grad is
    refused, here and in the calls below; one with a forward-mode tangent is
    always."""
    args = _rope_args(pos, axes, theta, style, eps, q, (q, None, q_out, q_weight, None),
                      (k, None, k_out, k_weight, None))
    status = lib().dit_rope_forward(args, _raw_stream(q, stream))
    if status:
        _check(status)


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
    L, s, ws, n, owner = lib(), _raw_stream(dq_out, stream), 0, 0, None
    if dq_weight is not None or dk_weight is not None:
        ws, n, owner = _workspace(dq_out, workspace, stream, L.dit_rope_workspace_bytes(args))
    _check(L.dit_rope_backward(args, ws, n, s))


def dit_rope_workspace_bytes(head_dim: int) -> int:
    """Workspace that is enough for any dit_rope_backward with weight gradients."""
    heads = (1, 0, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, 16, 32)
    none = (0, 0, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, 0, 0)
    try:
        args = _ROPE_ARGS.pack(1, 1 << 20, head_dim, DTYPE_F32, 0, 1, 0, 0, 0, 0, 1e4, 0.0, 0, 0, 0, POS_I32, 0, *heads, *none)
    except (struct.error, OverflowError) as e:
        _refuse_scalar(e)
    n = lib().dit_rope_workspace_bytes(args)
    if n < 0:
        raise DitError(DIT_ERR_SHAPE, lib().dit_last_error().decode())
    return n


def _pixel_view(name, t, shape, dtype):
    """(pointer, batch stride, pixel stride) of a [batch, ..., channels] view."""
    if t.shape != shape:
        _refuse(DIT_ERR_SHAPE, f"{name} is {list(t.shape)}, not {list(shape)}")
    if t.dtype is not dtype:
        _refuse(DIT_ERR_INVALID_ARG, f"{name} is {t.dtype}, not {dtype}")
    stride = t.stride()
    if t.numel() == 0:
        return 0, 0, 0
    if stride[-1] != 1 and shape[-1] > 1:
        _refuse(DIT_ERR_SHAPE, f"{name}: channels must be contiguous (channels last)")
    step = stride[-2]
    if len(shape) > 3:  # the middle axes as one axis of pixels
        step = span = None  # 0 is a stride like any other (expanded views)
        for i in range(len(shape) - 2, 0, -1):
            if shape[i] == 1:
                continue
            if step is None:
                step = stride[i]
            elif stride[i] != span:
                _refuse(DIT_ERR_SHAPE, f"{name}: the axes between batch and channels must have one common stride")
            span = stride[i] * shape[i]
        step = step or 0
    return t.data_ptr(), stride[0], step


def _gn_args(x, dy, out, groups, weight, bias, mean, rstd, dweight, dbias, eps, act):
    _torch or _use_torch()
    if out is not None and _grad_mode() and (x.requires_grad or weight is not None and weight.requires_grad or
                                             bias is not None and bias.requires_grad or
                                             dy is not None and dy.requires_grad):
        _refuse_autograd()
    if out is not None and _forward_ad._current_level >= 0:
        _refuse_tangents(x, weight, bias, dy, mean, rstd)
    shape, dtype = x.shape, x.dtype
    if len(shape) < 3:
        _refuse(DIT_ERR_SHAPE, "x must be [batch, ..., channels]")
    B, C, P = shape[0], shape[-1], 1
    for v in shape[1:-1]:
        P *= v
    try:
        return _GN_ARGS.pack(B, P, C, groups, _dtype_code(dtype), act, eps, 0, *_pixel_view("x", x, shape, dtype),
                             *((0, 0, 0) if dy is None else _pixel_view("dy", dy, shape, dtype)),
                             *((0, 0, 0) if out is None else _pixel_view("out", out, shape, dtype)),
                             _param("weight", weight, (C,)), _param("bias", bias, (C,)),
                             _param("mean", mean, (B, groups)), _param("rstd", rstd, (B, groups)),
                             _param("dweight", dweight, (C,)), _param("dbias", dbias, (C,)))
    except (struct.error, OverflowError) as e:
        _refuse_scalar(e)


def dit_group_norm_forward(x, y, groups: int, *, weight=None, bias=None, mean=None, rstd=None, eps=1e-6, act=ACT_NONE,
                           workspace=None, stream=None):
    """Group norm of x [batch, ..., channels] (channels last) with an
    activation, into y (which may be x).  mean / rstd: float32 [batch, groups]
    written for the backward call, or None.  workspace: a contiguous tensor of
    dit_group_norm_workspace_bytes, or None to take one from torch's allocator
    (only on torch's current stream)."""
    args = _gn_args(x, None, y, groups, weight, bias, mean, rstd, None, None, eps, act)
    L, s = lib(), _raw_stream(x, stream)
    ws, n, owner = _workspace(x, workspace, stream, L.dit_group_norm_workspace_bytes(args, 0))
    _check(L.dit_group_norm_forward(args, ws, n, s))


def dit_group_norm_backward(x, dy, mean, rstd, dx, groups: int, *, weight=None, bias=None, dweight=None, dbias=None,
                            act=ACT_NONE, workspace=None, stream=None):
    """Gradient of dit_group_norm_forward: dx (which may be dy or x), and
    dweight / dbias (float32 [channels], overwritten) where given.  mean and
    rstd are what the forward call wrote."""
    args = _gn_args(x, dy, dx, groups, weight, bias, mean, rstd, dweight, dbias, 0.0, act)
    L, s = lib(), _raw_stream(x, stream)
    ws, n, owner = _workspace(x, workspace, stream, L.dit_group_norm_workspace_bytes(args, 1))
    _check(L.dit_group_norm_backward(args, ws, n, s))


def dit_group_norm_workspace_bytes(x, groups: int, backward: bool) -> int:
    """Workspace of a group-norm call on tensors of x's shape and type."""
    n = lib().dit_group_norm_workspace_bytes(
        _gn_args(x, None, None, groups, None, None, None, None, None, None, 0.0, ACT_NONE), 1 if backward else 0)
    if n < 0:
        raise DitError(DIT_ERR_SHAPE, lib().dit_last_error().decode())
    return n


def _token_view(name, t, shape, dtype):
    """(pointer, batch stride, token stride) of a [..., channels] view: one axis in front of the channels is tokens of one
    batch element, of several the first is the batch."""
    if t is None:
        return 0, 0, 0
    if t.shape == shape and t.dtype is dtype and len(shape) == 3:
        sb, st, sc = t.stride()
        if sc == 1:
            return t.data_ptr(), sb, st
    if len(shape) >= 3:
        return _pixel_view(name, t, shape, dtype)
    if t.shape != shape or t.dtype is not dtype:
        _bad_view(name, t, shape, dtype)
    if t.numel() and t.stride(-1) != 1 and shape[-1] > 1:
        _refuse(DIT_ERR_SHAPE, f"{name}: channels must be contiguous")
    return (t.data_ptr(), 0, t.stride(0) if len(shape) == 2 else 0) if t.numel() else (0, 0, 0)


def _norm_rows(shape):
    """batch, tokens and channels of a [..., channels] shape"""
    if len(shape) == 3:
        return shape
    if len(shape) < 1:
        _refuse(DIT_ERR_SHAPE, "x must be [..., channels]")
    B, N = (shape[0] if len(shape) > 3 else 1), 1
    for v in shape[1:-1] if len(shape) > 3 else shape[:-1]:
        N *= v
    return B, N, shape[-1]


def _norm_args(x, residual, total, dy, out, out_dtype, scale, weight, dweight, eps):
    torch = _torch or _use_torch()
    if _grad_mode() and (x.requires_grad or residual is not None and residual.requires_grad or
                         weight is not None and weight.requires_grad or dy is not None and dy.requires_grad):
        _refuse_autograd()
    if _forward_ad._current_level >= 0:
        _refuse_tangents(x, residual, weight, dy)
    shape, dtype = x.shape, x.dtype
    B, N, C = _norm_rows(shape)
    code = _dtype_code(dtype)
    if out_dtype is not dtype and out_dtype is not torch.float8_e4m3fn:
        _refuse(DIT_ERR_INVALID_ARG, f"out is {out_dtype}: {dtype} or float8_e4m3fn is wanted")
    try:
        return _NORM_ARGS.pack(B, N, C, code, code if out_dtype is dtype else DTYPE_E4M3, eps,
                               *_token_view("x", x, shape, dtype), *_token_view("residual", residual, shape, dtype),
                               *_token_view("total", total, shape, dtype), *_token_view("dy", dy, shape, dtype),
                               *_token_view("out", out, shape, out_dtype),
                               0 if scale is None else _param("scale", scale, shape[:-1]),
                               0 if weight is None else _param("weight", weight, (C,)),
                               0 if dweight is None else _param("dweight", dweight, (C,)))
    except (struct.error, OverflowError) as e:
        _refuse_scalar(e)


def dit_rms_norm_forward(x, out, *, residual=None, total=None, weight=None, scale=None, eps=1e-6, stream=None):
    """RMS norm over the channels of x [..., channels], of x + residual where a
    residual is given: total (which may be x or residual) receives that sum.
    out: of x's type (and possibly x or residual itself), or float8_e4m3fn with
    scale, float32 x.shape[:-1]: out * scale is the norm."""
    args = _norm_args(x, residual, total, None, out, out.dtype, scale, weight, None, eps)
    status = lib().dit_rms_norm_forward(args, _raw_stream(x, stream))
    if status:
        _check(status)


def dit_rms_norm_backward(total, dout, dx, *, dtotal=None, weight=None, dweight=None, eps=1e-6, workspace=None,
                          stream=None):
    """Gradient of dit_rms_norm_forward: total is what the norm was of (the
    forward's total, or x without a residual), dtotal the gradient that reaches
    it from elsewhere.  dx is the gradient of x, and of residual too; dweight
    (float32 [channels], overwritten) is computed where given.  workspace: a
    contiguous tensor of dit_rms_norm_workspace_bytes, or None to take one from
    torch's allocator (only on torch's current stream)."""
    args = _norm_args(total, dtotal, None, dout, dx, dx.dtype, None, weight, dweight, eps)
    L, s, ws, n, owner = lib(), _raw_stream(total, stream), 0, 0, None
    if dweight is not None:
        ws, n, owner = _workspace(total, workspace, stream, L.dit_rms_norm_workspace_bytes(args))
    _check(L.dit_rms_norm_backward(args, ws, n, s))


def dit_rms_norm_workspace_bytes(total) -> int:
    """Workspace of a dit_rms_norm_backward with dweight on tensors of this shape and type."""
    _torch or _use_torch()
    code = _dtype_code(total.dtype)
    n = lib().dit_rms_norm_workspace_bytes(_NORM_ARGS.pack(*_norm_rows(total.shape), code, code, 0.0, *(0,) * 15, 0, 16, 32))
    if n < 0:
        raise DitError(DIT_ERR_SHAPE, lib().dit_last_error().decode())
    return n


def _matrix(name, t, shape, dtype):
    """(pointer, row stride) of a [..., columns] view whose leading axes have one common stride."""
    if t is None:
        return 0, 0
    if t.shape != shape or t.dtype is not dtype:
        _bad_view(name, t, shape, dtype)
    if len(shape) == 2:
        step, column = t.stride()
        if column == 1:
            return t.data_ptr(), step
    if t.numel() == 0:
        return 0, 0
    stride = t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        _refuse(DIT_ERR_SHAPE, f"{name}: the last axis must be contiguous")
    if len(shape) == 2:
        return t.data_ptr(), stride[0]
    step = span = None
    for i in range(len(shape) - 2, -1, -1):
        if shape[i] == 1:
            continue
        if step is None:
            step = stride[i]
        elif stride[i] != span:
            _refuse(DIT_ERR_SHAPE, f"{name}: the axes in front of the last must have one common stride")
        span = stride[i] * shape[i]
    return t.data_ptr(), step or 0


def _ffn_args(x, w_gate, w_up, out, gate, up, act, x_scale=None, gate_scale=None, up_scale=None, bias_gate=None,
              bias_up=None, dx=None, dw_gate=None, dw_up=None, dbias_gate=None, dbias_up=None):
    _torch or _use_torch()
    if _grad_mode() and (x.requires_grad or w_gate.requires_grad or w_up.requires_grad or
                         bias_gate is not None and bias_gate.requires_grad or
                         bias_up is not None and bias_up.requires_grad or
                         x_scale is not None and x_scale.requires_grad or
                         gate_scale is not None and gate_scale.requires_grad or
                         up_scale is not None and up_scale.requires_grad):
        _refuse_autograd()
    if _forward_ad._current_level >= 0:
        _refuse_tangents(x, w_gate, w_up, x_scale, gate_scale, up_scale, bias_gate, bias_up)
    xs, ws = x.shape, w_gate.shape
    if len(xs) < 1 or len(ws) != 2 or ws[1] != xs[-1]:
        _refuse(DIT_ERR_SHAPE, f"x is {list(xs)} and w_gate {list(ws)}: [..., width] and [hidden, width] are wanted")
    F, D = ws
    rows = 1
    for v in xs[:-1]:
        rows *= v
    hs, dtype, operand = xs[:-1] + (F,), out.dtype, x.dtype
    codes = _operand_codes.get(dtype), _operand_codes.get(operand)
    if None in codes:
        _refuse(DIT_ERR_INVALID_ARG, f"unsupported dtype {dtype if codes[0] is None else operand}")
    try:
        return _FFN_ARGS.pack(rows, D, F, *codes, act, 0, *_matrix("x", x, xs, operand), *_matrix("w_gate", w_gate, ws, operand),
                              *_matrix("w_up", w_up, ws, operand),
                              0 if x_scale is None else _param("x_scale", x_scale, xs[:-1]),
                              0 if gate_scale is None else _param("gate_scale", gate_scale, (F,)),
                              0 if up_scale is None else _param("up_scale", up_scale, (F,)),
                              0 if bias_gate is None else _param("bias_gate", bias_gate, (F,)),
                              0 if bias_up is None else _param("bias_up", bias_up, (F,)),
                              *_matrix("gate", gate, hs, dtype), *_matrix("up", up, hs, dtype),
                              *_matrix("out", out, hs, dtype), *_matrix("dx", dx, xs, dtype),
                              *_matrix("dw_gate", dw_gate, ws, dtype), *_matrix("dw_up", dw_up, ws, dtype),
                              0 if dbias_gate is None else _param("dbias_gate", dbias_gate, (F,)),
                              0 if dbias_up is None else _param("dbias_up", dbias_up, (F,)))
    except (struct.error, OverflowError) as e:
        _refuse_scalar(e)


def dit_gated_ffn_forward(x, w_gate, w_up, out, *, gate=None, up=None, bias_gate=None, bias_up=None, x_scale=None,
                          gate_scale=None, up_scale=None, act=ACT_SILU, workspace=None, stream=None):
    """out [..., hidden] = act(x w_gate^T + bias_gate) * (x w_up^T + bias_up) of x
    [..., width] and weights [hidden, width], in bfloat16 or float16.  gate / up
    receive the two projections, for the backward call.  With x and the weights
    in float8_e4m3fn, x_scale (float32 x.shape[:-1]) and gate_scale / up_scale
    (float32 [hidden]) make the values they stand for.  act: ACT_SILU or
    ACT_GELU (tanh form).  workspace: a contiguous tensor of
    dit_gated_ffn_workspace_bytes, or None to take one from torch's allocator
    where the call needs it (only on torch's current stream)."""
    args = _ffn_args(x, w_gate, w_up, out, gate, up, act, x_scale, gate_scale, up_scale, bias_gate, bias_up)
    L, s = lib(), _raw_stream(x, stream)
    ws, n, owner = _workspace(x, workspace, stream, L.dit_gated_ffn_workspace_bytes(args, 0))
    _check(L.dit_gated_ffn_forward(args, ws, n, s))


def dit_gated_ffn_backward(x, w_gate, w_up, gate, up, dout, *, dx=None, dw_gate=None, dw_up=None, dbias_gate=None,
                           dbias_up=None, act=ACT_SILU, workspace=None, stream=None):
    """Gradient of dit_gated_ffn_forward from the gate and up that it kept.  Each
    of dx, dw_gate, dw_up (of the inputs' type) and dbias_gate, dbias_up (float32
    [hidden]) is overwritten where given."""
    _torch or _use_torch()
    if (gate.requires_grad or up.requires_grad or dout.requires_grad) and _grad_mode():
        _refuse_autograd()
    if _forward_ad._current_level >= 0:
        _refuse_tangents(gate, up, dout)
    args = _ffn_args(x, w_gate, w_up, dout, gate, up, act, dx=dx, dw_gate=dw_gate, dw_up=dw_up, dbias_gate=dbias_gate,
                     dbias_up=dbias_up)
    L, s = lib(), _raw_stream(x, stream)
    ws, n, owner = _workspace(x, workspace, stream, L.dit_gated_ffn_workspace_bytes(args, 1))
    _check(L.dit_gated_ffn_backward(args, ws, n, s))


def dit_gated_ffn_workspace_bytes(x, w_gate, *, backward=False) -> int:
    """Workspace that is enough for any call on tensors of the shapes and types of x and w_gate, whatever their strides
    and alignment and whichever gradients are wanted."""
    torch = _torch or _use_torch()
    rows, most = x.numel() // max(1, x.shape[-1]), 0
    operand = _operand_codes.get(x.dtype, -1)
    code, p = DTYPE_BF16 if operand == DTYPE_E4M3 else operand, 16 + 1  # a pointer that needs a copy
    scale = 16 if operand == DTYPE_E4M3 else 0
    F, D = w_gate.shape
    # dx asks for its share beside the weights' gradients; one of these may split its rows where both would not
    for wanted in ((16, 16, 16), (16, 16, 0)) if backward else ((0, 0, 0),):
        n = lib().dit_gated_ffn_workspace_bytes(_FFN_ARGS.pack(
            rows, D, F, code, operand, ACT_SILU, 0, p, D, p, D, p, D, scale, scale, scale, 0, 0, 16, F, 16, F, 16, F,
            *(v for w in wanted for v in (w, D)), 16 * backward, 16 * backward), int(backward))
        if n < 0:
            raise DitError(DIT_ERR_SHAPE, lib().dit_last_error().decode())
        most = max(most, n)
    return most


def dit_gated_ffn_synchronize(stream=None):
    """Wait for the stream (of the current device) and raise if a gated feed-forward kernel abandoned a wait on it."""
    _check(lib().dit_gated_ffn_synchronize(_stream(stream)))


_dtype_of, _requires_grad_of = operator.attrgetter("dtype"), operator.attrgetter("requires_grad")


def _grad_tensors(grads, clipped):
    """The packed dit_grad_tensors of the entries that are not None, and their number."""
    T = (_torch or _use_torch()).Tensor
    live = [g for g in grads if g is not None]
    # whole lists at a time: a model has hundreds of gradients
    dtypes, sizes, pointers = list(map(_dtype_of, live)), list(map(T.numel, live)), list(map(T.data_ptr, live))
    codes = list(map(_dtype_codes.get, dtypes))
    if None in codes:
        _refuse(DIT_ERR_INVALID_ARG, f"a gradient is {dtypes[codes.index(None)]}")
    if not all(map(T.is_contiguous, live)):
        _refuse(DIT_ERR_SHAPE, "gradients must be contiguous")
    if _grad_mode() and any(map(_requires_grad_of, live)):
        _refuse_autograd()
    if _forward_ad._current_level >= 0:
        _refuse_tangents(*live)
    n = len(live)
    if clipped is None:
        outs = [0] * n
    elif clipped is grads:
        outs = pointers
    else:
        made = [c for c in clipped if c is not None]
        # None at the same places: an entry left out in only one list would shift all behind it
        if (len(clipped) != len(grads) or
                (n < len(grads) or len(made) < len(clipped)) and [g is None for g in grads] != [c is None for c in clipped] or
                list(map(T.numel, made)) != sizes or list(map(_dtype_of, made)) != dtypes or not all(map(T.is_contiguous, made))):
            _refuse(DIT_ERR_SHAPE, "clipped must hold a contiguous tensor of the size and type of each gradient at its place")
        outs = list(map(T.data_ptr, made))
    # structures of four 64-bit fields (the type and the reserved field as one)
    fields = array.array("q", bytes(32 * n))
    for i, column in enumerate((pointers, outs, sizes, codes)):
        fields[i::4] = array.array("q", column)
    return fields.tobytes(), n


def dit_grad_norm(grads, norm, *, max_norm=None, clipped=None, workspace=None, stream=None):
    """norm (a float32 CUDA tensor of one element) = the 2-norm of all tensors of
    the list `grads` together (None entries are left out).  With max_norm they
    are multiplied by max_norm / norm where norm is above it, in place or into
    the tensors at the same places of the list `clipped`; a norm that is not
    finite leaves the values as they are.  workspace: a contiguous tensor of
    dit_grad_norm_workspace_bytes, or None to take one from torch's allocator
    (only on torch's current stream)."""
    torch = _torch or _use_torch()
    if not isinstance(grads, (list, tuple)):
        grads = list(grads)
    limit = _INF
    if max_norm is None:
        if clipped is not None:
            _refuse(DIT_ERR_INVALID_ARG, "clipped without max_norm")
    else:
        try:
            limit = C.c_float(max_norm).value
        except TypeError as e:
            _refuse_scalar(e)
        if limit == _INF:
            _refuse(DIT_ERR_INVALID_ARG, "max_norm must be finite (None: the norm only)")
        if clipped is None:
            clipped = grads
        elif not isinstance(clipped, (list, tuple)):
            clipped = list(clipped)
    if norm.dtype is not torch.float32 or norm.numel() != 1:
        _refuse(DIT_ERR_INVALID_ARG, "norm must be one float32")
    tensors, n = _grad_tensors(grads, clipped)
    L, s = lib(), _raw_stream(norm, stream)
    ws, size, owner = _workspace(norm, workspace, stream, L.dit_grad_norm_workspace_bytes(tensors, n))
    _check(L.dit_grad_norm(tensors, n, limit, norm.data_ptr(), ws, size, s))


def dit_grad_norm_workspace_bytes(grads) -> int:
    """Workspace of a dit_grad_norm call on these tensors."""
    n = lib().dit_grad_norm_workspace_bytes(*_grad_tensors(grads, None))
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
