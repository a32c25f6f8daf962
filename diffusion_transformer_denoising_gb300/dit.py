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
_torch = None          # the module, its dtypes as dit.h names them and its grad mode, on first use
_dtype_codes = {}
_grad_mode = None


def _use_torch():
    global _torch, _grad_mode
    if _torch is None:
        import torch
        _grad_mode = torch.is_grad_enabled
        _dtype_codes.update({torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16})
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
    refused, here and in the calls below."""
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
