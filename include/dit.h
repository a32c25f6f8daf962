/*
 * dit.h -- C ABI of the GB300 denoiser stage (libdit.so).
 *
 * The denoiser stage runs the network's forward passes over the whole step
 * schedule, with the sampler advancing the latent after each of them
 * (SGLang-Diffusion "Disaggregated Diffusion Pipeline", Quick Start, role
 * table: "denoiser").  Its inputs are the latents, the
 * timestep / sigma schedule in the exact order used, the positive prompt
 * embeddings and, when classifier-free guidance is on, the negative ones
 * (SGLang-Diffusion "Support New Diffusion Models", section 4, table of the
 * fields DenoisingStage requires).  The network is called with
 * hidden_states / encoder_hidden_states / timestep, once with the positive
 * and once with the negative condition (same page, section 2 "Pipeline
 * Config").  Velocities are flow predictions integrated with a flow-matching
 * Euler step on a shifted sigma schedule (stable-diffusion.cpp "Model
 * Configuration Conventions", "Sampling And Geometry").
 *
 * Conventions for every call:
 *   - Every pointer documented "device" is a CUDA device pointer owned by the
 *     caller; the library never frees it.  Host pointers are read before the
 *     call returns.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Work is enqueued asynchronously on it; results are ready once
 *     the stream is synchronised (dit_synchronize does that and also reports
 *     a device-side timeout).
 *   - Argument errors are detected on the host before anything is launched;
 *     outputs are then left untouched.  Nothing aborts the process: every
 *     failure is a status code, with a message from dit_last_error().
 *   - There is no CPU fallback and no silent precision change: a call the
 *     GPU path cannot serve returns an error.
 *   - One model owns one device workspace that every forward call of that
 *     model reuses (block scratch, loop state, the timestep MLP's hidden
 *     activations).  Calls on the same model must therefore be ordered on
 *     the GPU: issue them on one stream, or order the streams with events.
 *     Calls of one model on two unordered streams race on the workspace.
 *     Separate models share nothing and may run concurrently.
 *   - Floating-point tensors crossing the ABI are float32, row-major, densely
 *     packed, in the layouts given per call (the operators beside the model
 *     take strided views of float32, bfloat16 or float16 activations).  B is
 *     the batch of network passes; in the loop B = 2 x requests with CFG
 *     (conditional passes first, then unconditional ones).
 */
#ifndef DIT_H
#define DIT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DIT_OK = 0,
  DIT_ERR_INVALID_ARG = 1, /* bad pointer, value, schedule or flag          */
  DIT_ERR_SHAPE = 2,       /* inconsistent or unsupported tensor shape      */
  DIT_ERR_NOT_LOADED = 3,  /* forward called before a complete weight load  */
  DIT_ERR_OOM = 4,         /* device allocation failed                      */
  DIT_ERR_CUDA = 5,        /* a CUDA runtime/driver call failed             */
  DIT_ERR_TIMEOUT = 6      /* a kernel gave up a bounded wait (see dit_synchronize) */
} dit_status;

enum { DIT_PREC_BF16 = 0, DIT_PREC_F32 = 1, DIT_PREC_FP8 = 2 };
enum { DIT_COND_CROSS = 0, DIT_COND_JOINT = 1 };
/* DIT_DTYPE_F16 and DIT_DTYPE_E4M3 are types of the operators beside the model
 * only: dit_load_weights takes the other two. */
enum { DIT_DTYPE_F32 = 0, DIT_DTYPE_BF16 = 1, DIT_DTYPE_F16 = 2, DIT_DTYPE_E4M3 = 3 };
/* dit_denoise_loop flags */
enum {
  DIT_LOOP_PARTIAL_SCHEDULE = 1, /* allow sigmas[0] != 1 or sigmas[n] != 0                     */
  DIT_LOOP_CUDA_GRAPH = 2        /* replay one captured step as a CUDA graph (see the loop call) */
};

/*
 * Model configuration, copied by dit_create.  Mirrors the C++ "*Config"
 * convention of stable-diffusion.cpp "Model Configuration Conventions"
 * (Config Types / Runner And Model Responsibilities): derived once, passed to
 * the model, never re-scanned.
 *   in_channels   latent channels C (stable-diffusion.cpp ModelGeometry latent_channels)
 *   patch[3]      patch size (pt, ph, pw) over (T, H, W) of the latent
 *   hidden        D = heads * head_dim
 *   mlp           F, width of the GELU MLP
 *   cond_dim      Dc, width of a condition token (must equal hidden in joint mode)
 *   freq_dim      width of the sinusoidal timestep embedding (even)
 *   rope_axes[3]  rotary channels per axis (t, h, w), each even, summing to
 *                 head_dim, or all zero for no rotation
 *   cond_mode     DIT_COND_CROSS: cross-attention to condition tokens;
 *                 DIT_COND_JOINT: dual-stream joint attention with them
 *   precision     DIT_PREC_BF16: bf16 weights/activations, fp32 accumulate
 *                 (tcgen05 tensor cores; requires head_dim == 128);
 *                 DIT_PREC_FP8: as bf16, except that the GEMMs fed by a
 *                 LayerNorm (self-attention Q/K/V, cross-attention Q, MLP
 *                 up-projection) take e4m3 operands: weights quantized at
 *                 load with one scale per output row, the LayerNorm output
 *                 with one scale per token row (requires hidden % 16 == 0);
 *                 DIT_PREC_F32: fp32 everywhere (test mode, CUDA cores)
 *   ln_eps, rope_theta, timestep_scale (t = timestep_scale * sigma)
 */
typedef struct {
  int32_t in_channels;
  int32_t patch[3];
  int32_t hidden;
  int32_t heads;
  int32_t head_dim;
  int32_t mlp;
  int32_t depth;
  int32_t cond_dim;
  int32_t freq_dim;
  int32_t rope_axes[3];
  int32_t cond_mode;
  int32_t precision;
  float ln_eps;
  float rope_theta;
  float timestep_scale;
} dit_config;

/* One named parameter for dit_load_weights.  `data` may be a host or a
 * device pointer (unified addressing decides); dtype is DIT_DTYPE_F32 or
 * DIT_DTYPE_BF16; shape[0..ndim) must equal the expected shape. */
typedef struct {
  const char* name;
  int32_t ndim;
  int64_t shape[4];
  int32_t dtype;
  const void* data;
} dit_tensor;

typedef struct dit_model dit_model;

/* Create a model on CUDA device `device`.  Validates the configuration
 * (DIT_ERR_INVALID_ARG / DIT_ERR_SHAPE) before touching the GPU. */
dit_status dit_create(const dit_config* cfg, int device, dit_model** out);

/* Copy parameters into the model's own device arena (converted to the
 * model's storage precision).  Strict: every name must be a known parameter,
 * appear once across all calls, and have the expected shape; otherwise
 * DIT_ERR_SHAPE and nothing of this call is kept (SGLang-Diffusion "Support
 * New Diffusion Models", "Reuse component loaders": strict key and shape
 * checks, fail instead of falling back).  The forward calls return
 * DIT_ERR_NOT_LOADED until every parameter has been loaded.  Synchronous.
 * With DIT_PREC_FP8 the weights of the self-attention Q/K/V, cross-attention
 * Q and MLP up-projection are quantized here on the device to e4m3 with one
 * scale per output row (max |row| / 448); the others are stored as bf16. */
dit_status dit_load_weights(dit_model* m, const dit_tensor* tensors, int n);

/* Host-only queries on a configuration (no GPU needed): the number of
 * parameters a model of this configuration expects, and the name (copied into
 * name_buf, NUL-terminated) and shape of the i-th, in load order.  Linear
 * weights are [out_features, in_features]; each block carries a learned
 * [6, hidden] modulation table (shift1, scale1, gate1, shift2, scale2,
 * gate2) added to the shared timestep modulation. */
int dit_num_params(const dit_config* cfg);
dit_status dit_param_info(const dit_config* cfg, int i, char* name_buf, int buf_len, int32_t* ndim,
                          int64_t shape[4]);

/* a1: timestep embedding -> MLP -> shared modulation.
 *   t_host  host float[batch], the network timestep per batch element
 *   mod     device float[batch, 6*hidden] output */
dit_status dit_timestep_modulation(dit_model* m, const float* t_host, int batch, float* mod, void* stream);

/* The same computation as dit_timestep_modulation, for callers that must
 * not allocate device memory during the call: for example a serving thread
 * that may not trigger the implicit device synchronisation a cudaMalloc or
 * cudaFree can cause, or a host whose device memory is entirely handed to
 * its own pool allocator, so any allocation by this library would fail or
 * stall.  (The pages have no counterpart; this is an interface addition.)
 * The call allocates nothing: it never calls cudaMalloc, cudaFree or any
 * allocating library routine, and it loads no module.  Its scratch (the
 * timesteps and the MLP's hidden activations) lives in one fixed array of
 * this library's device memory (about 1 MiB), which every GPU that loads the
 * library holds until the process exits.
 *   batch <= DIT_NOALLOC_MAX_BATCH, batch * hidden <= DIT_NOALLOC_MAX_HIDDEN,
 *   and hidden, freq_dim <= 12288 (one activation vector held in 48 KB of
 *   shared memory); otherwise DIT_ERR_INVALID_ARG (nothing is launched).
 * Set-up happens in dit_create, with the model's device current: it looks up
 * the array's device address on that device and loads the kernels this call
 * launches.  So create the model before any stream capture.  All calls share
 * the one array: calls whose work overlaps on the GPU (for example on two
 * streams without ordering between them) race with each other.  Every byte
 * of scratch a call reads it has written itself first. */
enum { DIT_NOALLOC_MAX_BATCH = 64, DIT_NOALLOC_MAX_HIDDEN = 262144 };
dit_status dit_timestep_modulation_noalloc(dit_model* m, const float* t_host, int batch, float* mod, void* stream);

/* a2: patchify + patch embedding.
 *   latents device float[batch, C, T, H, W]; latent_thw = {T, H, W}, each
 *           divisible by the patch size (else DIT_ERR_SHAPE)
 *   x       device float[batch, N, hidden] output, N = (T/pt)(H/ph)(W/pw),
 *           tokens in row-major (t, h, w) grid order */
dit_status dit_patch_embed(dit_model* m, const float* latents, int batch, const int32_t latent_thw[3],
                           float* x, void* stream);

/* a3-a9: one DiT block, in place on the residual stream(s).  The network
 * call of the pages (hidden_states = x, encoder_hidden_states = cond or xc,
 * the timestep through `mod`: SGLang-Diffusion "Support New Diffusion
 * Models", section 2 "Pipeline Config"), restricted to one block; rotary
 * positions follow the token grid ("Verify the Port": rotary shape and style
 * must match).
 *   block   0 .. depth-1
 *   x       device float[batch, N, hidden], image/video token stream, in/out
 *   xc      joint mode: device float[batch, cond_len, hidden], condition-token
 *           stream, in/out; cross mode: must be NULL
 *   mod     device float[batch, 6*hidden], the shared timestep modulation from
 *           dit_timestep_modulation (the block adds its own table)
 *   cond    cross mode: device float[batch, cond_len, cond_dim] condition
 *           tokens; joint mode: must be NULL
 *   grid    token grid {T/pt, H/ph, W/pw} (N = product), sets RoPE positions */
dit_status dit_block_forward(dit_model* m, int block, float* x, float* xc, const float* mod,
                             const float* cond, int batch, const int32_t grid[3], int cond_len,
                             void* stream);

/* a10: final layer (LN + head modulation + linear) and unpatchify.
 *   x  device float[batch, N, hidden];  mod as above
 *   v  device float[batch, C, T, H, W] output velocity */
dit_status dit_final_layer(dit_model* m, const float* x, const float* mod, int batch,
                           const int32_t latent_thw[3], float* v, void* stream);

/* a11 (first half): classifier-free guidance v = vu + g (vc - vu) over n
 * floats (device pointers; v may alias vc or vu).  The positive and negative
 * passes and the guidance scale: SGLang-Diffusion "Support New Diffusion
 * Models", section 1 "Sampling Params" (guidance_scale) and section 2
 * "Pipeline Config" (pos/neg kwargs).  n < 0, a NULL pointer with n > 0 or a
 * non-finite g: DIT_ERR_INVALID_ARG. */
dit_status cfg_combine(const float* vc, const float* vu, float g, float* v, int64_t n, void* stream);

/* a11 (second half): flow-matching Euler update x += (sigma_next - sigma) v
 * over n floats, in place on device x.  Flow prediction integrated on the
 * shifted sigma schedule: stable-diffusion.cpp "Model Configuration
 * Conventions", "Sampling And Geometry" (flow prediction, default flow
 * shift, flow denoisers).  n < 0, a NULL pointer with n > 0 or a non-finite
 * sigma: DIT_ERR_INVALID_ARG. */
dit_status flow_euler_step(float* x, const float* v, float sigma, float sigma_next, int64_t n,
                           void* stream);

/* ---------------------------------------------------------------------------
 * Operators beside the model: what a block around the denoiser's own needs on
 * its token grids and latents, forward and gradient.  They hold no state and
 * allocate nothing; scratch is the caller's `workspace` (device memory,
 * 16-byte aligned, its size from the ..._workspace_bytes call, contents
 * meaningless before and after).  Calls that share a workspace must be
 * ordered on the GPU, captured graphs among them.  Every pointer is a device
 * pointer of one device; the launch goes to that device whichever is current,
 * and `stream` must belong to it.  Results are the same bits from run to run.
 * The output `out` may be the very view (same pointer, same strides) of the x
 * or dy it is computed from.  Apart from that no output (dweight, dbias, the
 * forward's mean and rstd and the workspace among them) has a byte in common
 * with an input or another output: such calls are refused.  (Views of one
 * buffer whose strides do not nest are compared by a bounded search and may
 * pass unseen.)  A size of zero is a valid call.
 */

/* Rotary position embedding of q and k over 1 to 4 position axes (time,
 * height, width, ...), with an optional RMS norm of every head in front of it.
 * The rotary shape and style are named among the failure points of
 * SGLang-Diffusion "Support New Diffusion Models", "Verify the Port".
 *
 * R = axes[0] + ... channels of each head are turned as R / 2 pairs; axis a
 * owns axes[a] / 2 consecutive pairs, and its j-th pair of a token at
 * position pos[a] turns by pos[a] * theta^(-2 j / axes[a]).  Pair p is
 * channels (2p, 2p + 1) with DIT_ROPE_INTERLEAVED, (p, p + R / 2) with
 * DIT_ROPE_SPLIT; (a, b) -> (a cos - b sin, a sin + b cos).  Channels from R
 * on are not turned.  The angle pos * frequency is reduced exactly (64-bit
 * fixed-point turns); the frequency is good to 2^-53 of itself + 2^-55, so an
 * angle a is off by at most |a| 2^-53 + |pos| 2^-55 radians: cos and sin have
 * fp32 accuracy at every int32 position, 1e-4 at 2^40, none from 2^53 on.
 * With a weight w[head_dim] the head x is first x * w / sqrt(mean(x^2) + eps),
 * the mean over the whole head.
 * Arithmetic is fp32, rounded once to the activation type.  */
enum { DIT_ROPE_INTERLEAVED = 0, DIT_ROPE_SPLIT = 1 };
enum { DIT_ROPE_MAX_AXES = 4, DIT_ROPE_MAX_HEAD_DIM = 256 };
enum { DIT_POS_I32 = 0, DIT_POS_F32 = 1 };

/* One of the two tensors turned, as views [batch, tokens, heads, head_dim]
 * whose last axis is contiguous; strides in elements, of the batch, token and
 * head axes.  Inputs may have strides of 0 (expanded views). */
typedef struct {
  int32_t heads;         /* 0: tensor absent                                            */
  int32_t reserved;      /* 0                                                           */
  const void* x;         /* forward input (backward: needed with a weight, else unread) */
  int64_t x_stride[3];
  const void* dy;        /* backward: gradient of the forward output                    */
  int64_t dy_stride[3];
  void* out;             /* forward: output; backward: gradient of x                    */
  int64_t out_stride[3];
  const float* weight;   /* device float[head_dim] of the head norm, or NULL: no norm   */
  float* dweight;        /* backward: device float[head_dim], or NULL: not wanted       */
} dit_rope_heads;

typedef struct {
  int64_t batch;
  int64_t tokens;
  int32_t head_dim;      /* even, at most DIT_ROPE_MAX_HEAD_DIM                          */
  int32_t dtype;         /* DIT_DTYPE_* of x, dy and out                                */
  int32_t style;         /* DIT_ROPE_*                                                  */
  int32_t n_axes;        /* 1 .. DIT_ROPE_MAX_AXES                                      */
  int32_t axes[4];       /* channels per axis: even, >= 0, at most head_dim in all      */
  float theta;           /* >= 1                                                        */
  float eps;             /* >= 0                                                        */
  const void* pos;       /* device [batch, tokens, n_axes], last axis contiguous        */
  int64_t pos_stride[2]; /* batch (0: shared by the batch) and token strides, elements  */
  int32_t pos_dtype;     /* DIT_POS_I32, or DIT_POS_F32 (finite; else that token is NaN)  */
  int32_t reserved;      /* 0                                                           */
  dit_rope_heads q, k;   /* their head counts are independent                           */
} dit_rope_args;

dit_status dit_rope_forward(const dit_rope_args* a, void* stream);
/* out = the gradient of x; dweight = the gradient of the weight, summed over
 * batch, tokens and heads in fp32 (overwritten; all zero for no tokens).
 * Needs workspace when a dweight is wanted, unless the rows are few. */
dit_status dit_rope_backward(const dit_rope_args* a, void* workspace, int64_t workspace_bytes, void* stream);
/* Bytes dit_rope_backward needs (host-only query; pointers are read as
 * present or NULL only); -1 for arguments the call would refuse. */
int64_t dit_rope_workspace_bytes(const dit_rope_args* a);

/* Group norm of channels-last activations with an activation behind it: the
 * normalisation of the latent encoders and decoders on either side of the
 * denoiser (SGLang-Diffusion "Disaggregated Diffusion Pipeline", Quick Start,
 * role table: encoder, decoder).  x is a view [batch, pixels, channels] whose
 * last axis is contiguous (pixels = H W or T H W); strides in elements, of
 * the batch and pixel axes.  Each batch element's `groups` groups of
 * channels / groups consecutive channels are normalised over all pixels with
 * their mean and population variance, then y = act(xhat * weight + bias) per
 * channel.  Statistics and arithmetic are fp32, rounded once to the type.  */
enum { DIT_ACT_NONE = 0, DIT_ACT_SILU = 1, DIT_ACT_GELU = 2 };  /* GELU (tanh form): dit_gated_ffn_* only */
typedef struct {
  int64_t batch;
  int64_t pixels;
  int32_t channels;
  int32_t groups;       /* divides channels                                               */
  int32_t dtype;        /* DIT_DTYPE_* of x, dy and out                                  */
  int32_t act;          /* DIT_ACT_*                                                     */
  float eps;            /* >= 0; forward only                                            */
  int32_t reserved;     /* 0                                                             */
  const void* x;
  int64_t x_stride[2];
  const void* dy;       /* backward: gradient of the forward output                      */
  int64_t dy_stride[2];
  void* out;            /* forward: y; backward: gradient of x                           */
  int64_t out_stride[2];
  const float* weight;  /* device float[channels], or NULL: 1                            */
  const float* bias;    /* device float[channels], or NULL: 0                            */
  float* mean;          /* device float[batch, groups]: forward writes them (NULL: not   */
  float* rstd;          /*   wanted); backward reads what the forward wrote              */
  float* dweight;       /* backward: device float[channels], or NULL: not wanted         */
  float* dbias;         /* backward: device float[channels], or NULL: not wanted         */
} dit_group_norm_args;

/* With no pixels, mean is 0 and rstd 1 / sqrt(eps). */
dit_status dit_group_norm_forward(const dit_group_norm_args* a, void* workspace, int64_t workspace_bytes,
                                  void* stream);
/* dweight and dbias are sums over batch and pixels in fp32 (overwritten). */
dit_status dit_group_norm_backward(const dit_group_norm_args* a, void* workspace, int64_t workspace_bytes,
                                   void* stream);
/* Bytes of workspace of the forward (backward == 0) or the backward call
 * (host-only query, from the sizes and the type alone: enough for any strides
 * and alignment); -1 for arguments the call would refuse. */
int64_t dit_group_norm_workspace_bytes(const dit_group_norm_args* a, int backward);

/* RMS norm of channels-last activations with the residual's addition in front
 * of it: the feed-forward half of a block beside the denoiser's own (norm, then
 * dit_gated_ffn_forward).  x, residual, total and out are views [batch, tokens,
 * channels] whose last axis is contiguous; strides in elements, of the batch and
 * token axes.
 *   total = x + residual, rounded once to the type (total = x without residual)
 *   y = total * weight / sqrt(mean(total^2) + eps), the mean over the channels
 * out holds y in the type of x, or in e4m3 with a scale for each row: scale =
 * max |y| / 448 (1 for a row of zeros, at least 2^-126), out = y / scale rounded
 * to nearest even.  Such a row with a NaN or an infinity in it gets the scale NaN
 * and zeros.  The outputs total and out may be the very view of x or of residual
 * (out only in the type of x).  Arithmetic is fp32, the squares' sum too: a row
 * with values of 1e19 and more counts as one of infinite norm, its y is 0; squares
 * of values below 1e-19 lose digits, which an eps as small does not hide.  The
 * gradient of a row past 1e19 is dtotal alone, or NaN where the sum of weight *
 * total * dy overflows. */
enum { DIT_RMS_NORM_MAX_CHANNELS = 16384 };
typedef struct {
  int64_t batch;
  int64_t tokens;
  int32_t channels;      /* 1 .. DIT_RMS_NORM_MAX_CHANNELS                               */
  int32_t dtype;         /* DIT_DTYPE_F32, _BF16, _F16                                   */
  int32_t out_dtype;     /* forward: dtype, or DIT_DTYPE_E4M3; backward: dtype           */
  float eps;             /* >= 0                                                         */
  const void* x;         /* forward: input; backward: what the norm was of (the forward's total) */
  int64_t x_stride[2];
  const void* residual;  /* forward: or NULL; backward: the gradient that reaches total from elsewhere, or NULL */
  int64_t residual_stride[2];
  void* total;           /* forward: x + residual, or NULL: not wanted (NULL without residual); backward: NULL */
  int64_t total_stride[2];
  const void* dy;        /* backward: gradient of the forward's out                      */
  int64_t dy_stride[2];
  void* out;             /* forward: y; backward: the gradient of x, which is that of residual too */
  int64_t out_stride[2];
  float* scale;          /* out_dtype e4m3: device float[batch, tokens], dense; else NULL */
  const float* weight;   /* device float[channels], or NULL: 1                           */
  float* dweight;        /* backward: device float[channels], or NULL: not wanted        */
} dit_rms_norm_args;

dit_status dit_rms_norm_forward(const dit_rms_norm_args* a, void* stream);
/* dweight is the sum over batch and tokens in fp32 (overwritten; zero for no
 * rows) and needs workspace.  out may be the very view of x, residual or dy. */
dit_status dit_rms_norm_backward(const dit_rms_norm_args* a, void* workspace, int64_t workspace_bytes, void* stream);
/* Bytes dit_rms_norm_backward needs (host-only query; pointers are read as
 * present or NULL only); -1 for arguments the call would refuse. */
int64_t dit_rms_norm_workspace_bytes(const dit_rms_norm_args* a);

/* Gated feed-forward: both projections, the activation and the product,
 *   gate = x w_gate^T + bias_gate,  up = x w_up^T + bias_up,
 *   out = act(gate) * up
 * with act SiLU or GELU (tanh form), where the denoiser's own MLP has one
 * projection and GELU.  x is [rows, width], the weights [hidden, width], out,
 * gate and up [rows, hidden], all with a contiguous last axis and one stride in
 * elements.  dtype is that of out, gate and up, and (operand_dtype ==
 * dtype) of x and the weights.  With operand_dtype DIT_DTYPE_E4M3, x and the
 * weights are e4m3, x * x_scale[row] and w * scale[channel] the values they
 * stand for; forward only.  A sum is multiplied by the channel's scale, then by
 * the row's: any normal number as x_scale, 2^-100 to 2^90 as the others keep all
 * its digits.  Sums are fp32 on the tensor cores, every output is rounded once.  No
 * output has a byte in common with an input.  Operands whose pointer or stride is
 * no multiple of 16 bytes are copied into the workspace first, but for up to 32
 * rows in the forward call. */
typedef struct {
  int64_t rows;
  int32_t width;             /* 1 .. 2^17                                                   */
  int32_t hidden;            /* 1 .. 2^17                                                   */
  int32_t dtype;             /* DIT_DTYPE_BF16 or DIT_DTYPE_F16                             */
  int32_t operand_dtype;     /* dtype, or DIT_DTYPE_E4M3 (forward)                          */
  int32_t act;               /* DIT_ACT_SILU or DIT_ACT_GELU                                */
  int32_t reserved;          /* 0                                                           */
  const void* x;
  int64_t x_stride;
  const void* w_gate;
  int64_t w_gate_stride;
  const void* w_up;
  int64_t w_up_stride;
  const float* x_scale;      /* e4m3: device float[rows]; else NULL                         */
  const float* gate_scale;   /* e4m3: device float[hidden]; else NULL                       */
  const float* up_scale;     /* e4m3: device float[hidden]; else NULL                       */
  const float* bias_gate;    /* forward: device float[hidden], or NULL: 0                   */
  const float* bias_up;      /* forward: device float[hidden], or NULL: 0                   */
  void* gate;                /* forward: kept for the backward call, or NULL; backward: read */
  int64_t gate_stride;
  void* up;                  /* as gate; both or neither                                    */
  int64_t up_stride;
  void* out;                 /* forward: output; backward: the output's gradient, read      */
  int64_t out_stride;
  void* dx;                  /* backward: gradient of x, or NULL: not wanted                */
  int64_t dx_stride;
  void* dw_gate;             /* backward: gradients of the weights, or NULL: not wanted     */
  int64_t dw_gate_stride;
  void* dw_up;
  int64_t dw_up_stride;
  float* dbias_gate;         /* backward: device float[hidden], or NULL: not wanted         */
  float* dbias_up;
} dit_gated_ffn_args;

dit_status dit_gated_ffn_forward(const dit_gated_ffn_args* a, void* workspace, int64_t workspace_bytes, void* stream);
/* The gradient from the gate and up that the forward call kept.  The gradients
 * of gate and up are formed in fp32, summed into dbias_* as they are, and
 * rounded to dtype as operands of the products (in fp16 those above 65504 become
 * infinite and those below 6e-5 lose digits, as between separate calls: a scaled
 * loss keeps them in range); dx, dw_gate and dw_up are fp32 sums rounded to dtype
 * (overwritten; zero for no rows). */
dit_status dit_gated_ffn_backward(const dit_gated_ffn_args* a, void* workspace, int64_t workspace_bytes, void* stream);
/* Bytes of workspace of the forward (backward == 0) or the backward call
 * (host-only query; pointers are read as present, NULL or aligned only);
 * -1 for arguments the call would refuse. */
int64_t dit_gated_ffn_workspace_bytes(const dit_gated_ffn_args* a, int backward);
/* Synchronise `stream`, a stream of the current device, and report
 * DIT_ERR_TIMEOUT if a kernel of dit_gated_ffn_* on that device abandoned a
 * bounded wait since the last check (its outputs are then invalid). */
dit_status dit_gated_ffn_synchronize(void* stream);

/* The norm of many tensors together (the gradients of a model, after a
 * backward pass), and their clipping to it:
 *   norm = sqrt(sum of all squares),
 *   out = grad * (norm > max_norm ? max_norm / norm : 1), rounded once.
 * Tensors are dense, of one type each.  A tensor's out may be the very grad
 * (then nothing is written unless the norm is above max_norm); all are NULL
 * when max_norm is infinite: the norm only.  A norm that is NaN or infinite
 * leaves the values as they are: the caller learns of it by the norm.  Squares
 * are summed in fp32 over a few dozen values and in fp64 from there, and do not
 * overflow. */
typedef struct {
  const void* grad;
  void* out;
  int64_t numel;
  int32_t dtype;         /* DIT_DTYPE_F32, _BF16 or _F16 */
  int32_t reserved;      /* 0 */
} dit_grad_tensor;
/* tensors: host array of n entries, read before the call returns; max_norm >= 0;
 * norm: device float.  workspace of dit_grad_norm_workspace_bytes. */
dit_status dit_grad_norm(const dit_grad_tensor* tensors, int64_t n, float max_norm, float* norm, void* workspace,
                         int64_t workspace_bytes, void* stream);
int64_t dit_grad_norm_workspace_bytes(const dit_grad_tensor* tensors, int64_t n);

/* The whole denoiser stage for `batch` requests: the denoiser role of
 * SGLang-Diffusion "Disaggregated Diffusion Pipeline" (Quick Start, role
 * table), with the inputs that "Support New Diffusion Models" section 4 lists
 * for the denoising stage (latents, the sigma schedule in the order used,
 * positive and negative condition embeddings, number of steps); the error
 * cases follow that page's "Verify the Port" failure points (reversed
 * timesteps, missing negative embeddings with CFG on, latent shape).
 *   latents  device float[batch, C, T, H, W], initial noise in, denoised out
 *   cond     device float[batch, cond_len, cond_dim] positive condition
 *   uncond   device float[batch, cond_len, cond_dim] negative condition, or
 *            NULL for no guidance (then `guidance` must be 1)
 *   sigmas   host float[n_steps + 1], already shifted, strictly decreasing,
 *            sigmas[0] == 1 and sigmas[n_steps] == 0 unless
 *            DIT_LOOP_PARTIAL_SCHEDULE is set (resuming part of a schedule)
 *   Per step i: t = timestep_scale * sigmas[i]; v from the network on the
 *   2*batch conditional+unconditional passes; v = vu + g (vc - vu);
 *   latents += (sigmas[i+1] - sigmas[i]) v.  Condition-token keys/values of
 *   cross-attention are computed once per call (they do not depend on the
 *   step). */
/*   With DIT_LOOP_CUDA_GRAPH the launches of one step are captured once (on
 *   a stream the model owns; nothing runs during the capture) into a CUDA
 *   graph that is then launched n_steps times on `stream`.  Every step reads
 *   its timestep and Euler increment from a device copy of `sigmas` through a
 *   device step counter, so the same graph serves every step; the result is
 *   bitwise the same as without the flag.  The graph is kept in the model and
 *   reused by later calls whose pointers, shapes, guidance and n_steps are
 *   the same; otherwise it is captured again.  Cannot be combined with
 *   per-launch timing (dit_profile_start with timing on): DIT_ERR_INVALID_ARG. */
dit_status dit_denoise_loop(dit_model* m, float* latents, int batch, const int32_t latent_thw[3],
                            const float* cond, const float* uncond, int cond_len,
                            const float* sigmas, int n_steps, float guidance, uint32_t flags,
                            void* stream);

/* Synchronise `stream` and report DIT_ERR_TIMEOUT if a kernel of this model
 * abandoned a bounded wait since the last check (its outputs are then
 * invalid; the flag is cleared). */
dit_status dit_synchronize(dit_model* m, void* stream);

/* Per-kernel accounting of this model's launches, for measurement.
 * dit_profile_start resets the counters and, when `timing` is non-zero,
 * records a CUDA event pair on the launching stream around every launch.
 * dit_profile_stop synchronises the device and returns, per kernel kind,
 * the number of kernel launches and (with timing) their summed device time
 * in milliseconds.  counts/ms: host arrays of DIT_KERNEL_KINDS entries. */
enum {
  DIT_KERNEL_GEMM_QKV = 0,    /* self-attention Q/K/V projection (+RoPE scatter)  */
  DIT_KERNEL_GEMM_OUT = 1,    /* attention output projections (gated residual)   */
  DIT_KERNEL_GEMM_CROSS_Q = 2,
  DIT_KERNEL_GEMM_CROSS_KV = 3,
  DIT_KERNEL_GEMM_FFN1 = 4,   /* MLP up-projection + GELU                         */
  DIT_KERNEL_GEMM_FFN2 = 5,   /* MLP down-projection (gated residual)             */
  DIT_KERNEL_GEMM_EMBED = 6,  /* patch embedding and final linear                 */
  DIT_KERNEL_ATTN_SELF = 7,
  DIT_KERNEL_ATTN_CROSS = 8,
  DIT_KERNEL_LN = 9,          /* LayerNorm + adaLN modulation                     */
  DIT_KERNEL_SMALL = 10,      /* timestep MLP, tables, packing, casts             */
  DIT_KERNEL_CFG_EULER = 11,  /* guidance + Euler update of the loop              */
  DIT_KERNEL_KINDS = 12
};
dit_status dit_profile_start(dit_model* m, int timing);
dit_status dit_profile_stop(dit_model* m, int64_t* counts, double* ms);

/* Bytes of device memory held by the model (weights + workspace). */
int64_t dit_device_bytes(const dit_model* m);

void dit_destroy(dit_model* m);
const char* dit_status_string(dit_status s);
/* Message of the last failing call on this thread ("" if none). */
const char* dit_last_error(void);

/* Test hook: make the next `n`-th device allocation of any model fail with
 * DIT_ERR_OOM (0 disables).  Host-side only; used to test failure paths. */
void dit_debug_fail_alloc_after(int n);

/* Test hook: where GEMMs whose output width is a multiple of 256 run on
 * clusters of two CTAs that share one tcgen05.mma of 256 x 256
 * (cta_group::2) instead of single CTAs with 128 x 256 tiles.  mode 1 (the
 * default): when the GEMM's main loop has at least 16 K blocks (K >= 1024 in
 * bf16, K >= 2048 in e4m3); 0: never; 2: always.  Other values are clamped
 * to 0..2.  Process-wide; takes effect at the next launch (a CUDA graph
 * captured before keeps the kernels it captured).  Both paths give the same
 * bits; the hook exists to compare them. */
void dit_debug_gemm_cta_pairs(int mode);

/* Test hook for the device-side failure path.  Enqueues on `stream` a kernel
 * whose bounded wait on a barrier that nothing ever arrives on gives up after
 * the library's wait limit (1.5 s) and records DIT_DEBUG_STALL_SITE in the
 * model's error word; the next dit_synchronize then returns DIT_ERR_TIMEOUT
 * (and clears the word).  Nothing faults or hangs, and the model stays
 * usable.  Returns DIT_ERR_INVALID_ARG for a NULL model, DIT_ERR_CUDA if the
 * launch fails. */
enum { DIT_DEBUG_STALL_SITE = 99 };
dit_status dit_debug_stall(dit_model* m, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DIT_H */
