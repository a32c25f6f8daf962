// C ABI of the operators of a gated feed-forward block (RMS norm with residual,
// gated feed-forward, gradient norm): argument checks on the host, then the
// launch on the device that owns the tensors.
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "operator_checks.h"
#include "operators.h"
#include "tmap.h"

using namespace dit;

// the binding packs these structures by hand
static_assert(sizeof(dit_rms_norm_args) == 176 && sizeof(dit_gated_ffn_args) == 232 && sizeof(dit_grad_tensor) == 32,
              "layout of the ABI structures");

namespace {

bool activation_type(int dtype) { return dtype == DIT_DTYPE_F32 || dtype == DIT_DTYPE_BF16 || dtype == DIT_DTYPE_F16; }

// ---------------------------------------------------------------- rms norm
dit_status check_norm_shape(const dit_rms_norm_args* a, bool backward) {
  if (!a) return fail(DIT_ERR_INVALID_ARG, "arguments are NULL");
  if (a->batch < 0 || a->tokens < 0) return fail(DIT_ERR_SHAPE, "negative batch or tokens");
  if (a->batch > INT32_MAX || a->tokens > INT32_MAX || a->batch * a->tokens > INT32_MAX)
    return fail(DIT_ERR_SHAPE, "batch * tokens must be below 2^31");
  if (a->channels <= 0 || a->channels > DIT_RMS_NORM_MAX_CHANNELS)
    return fail(DIT_ERR_SHAPE, "channels must be 1 .. %d", DIT_RMS_NORM_MAX_CHANNELS);
  if (!activation_type(a->dtype)) return fail(DIT_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
  if (a->out_dtype != a->dtype && (backward || a->out_dtype != DIT_DTYPE_E4M3))
    return fail(DIT_ERR_INVALID_ARG, backward ? "out_dtype must be dtype" : "out_dtype must be dtype or e4m3");
  if (!(a->eps >= 0.f) || !isfinite(a->eps)) return fail(DIT_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (backward ? a->scale != nullptr : (a->scale == nullptr) == (a->out_dtype == DIT_DTYPE_E4M3) && a->batch * a->tokens)
    return fail(DIT_ERR_INVALID_ARG, "scale belongs to an output in e4m3, which needs it");
  if (!backward && (a->dy || a->dweight)) return fail(DIT_ERR_INVALID_ARG, "dy and dweight belong to the backward call");
  if (backward && a->total) return fail(DIT_ERR_INVALID_ARG, "the backward call reads the forward's total as x");
  if (!a->residual && a->total) return fail(DIT_ERR_INVALID_ARG, "total without residual is x");
  if (a->dweight && !a->weight) return fail(DIT_ERR_INVALID_ARG, "dweight without weight");
  return DIT_OK;
}

dit_status norm_call(const dit_rms_norm_args* a, bool backward, void* ws, int64_t ws_bytes, cudaStream_t stream) {
  clear_last_error();
  DIT_TRY(check_norm_shape(a, backward));
  const int elem = elem_bytes(a->dtype), out_elem = a->out_dtype == DIT_DTYPE_E4M3 ? 1 : elem;
  const int64_t size[2] = {a->batch, a->tokens}, rows = a->batch * a->tokens;
  const char* res_name = backward ? "dtotal" : "residual";
  if (rows) {
    DIT_TRY(check_view("x", a->x, 2, size, a->x_stride, a->channels, elem, false));
    if (a->residual) DIT_TRY(check_view(res_name, a->residual, 2, size, a->residual_stride, a->channels, elem, false));
    if (a->total) DIT_TRY(check_view("total", a->total, 2, size, a->total_stride, a->channels, elem, true));
    if (backward) DIT_TRY(check_view("dy", a->dy, 2, size, a->dy_stride, a->channels, elem, false));
    DIT_TRY(check_view("out", a->out, 2, size, a->out_stride, a->channels, out_elem, true));
    if (out_elem == elem) {
      DIT_TRY(check_in_place("x", a->x, a->x_stride, a->out, a->out_stride, size, 2));
      DIT_TRY(check_in_place(res_name, a->residual, a->residual_stride, a->out, a->out_stride, size, 2));
      if (backward) DIT_TRY(check_in_place("dy", a->dy, a->dy_stride, a->out, a->out_stride, size, 2));
    }
    if (a->total) {
      DIT_TRY(check_in_place("x", a->x, a->x_stride, a->total, a->total_stride, size, 2));
      DIT_TRY(check_in_place(res_name, a->residual, a->residual_stride, a->total, a->total_stride, size, 2));
    }
  }
  if (((uintptr_t)a->weight | (uintptr_t)a->dweight | (uintptr_t)a->scale) % 4)
    return fail(DIT_ERR_INVALID_ARG, "weights and scales must be aligned to 4 bytes");
  if (!rows && !a->dweight) return DIT_OK;
  const int64_t need = backward ? rms_norm_workspace(*a) : 0;
  DIT_TRY(check_workspace(ws, ws_bytes, need));
  Regions all;
  if (rows) {
    const int out = all.add("out", a->out, 2, size, a->out_stride, a->channels, out_elem, true);
    const int total = all.add("total", a->total, 2, size, a->total_stride, a->channels, elem, true);
    const int x = all.add("x", a->x, 2, size, a->x_stride, a->channels, elem, false);
    const int res = all.add(res_name, a->residual, 2, size, a->residual_stride, a->channels, elem, false);
    const int dy = backward ? all.add("dy", a->dy, 2, size, a->dy_stride, a->channels, elem, false) : -1;
    if (out_elem == elem)
      for (int in : {x, res, dy}) all.may_share(out, in);
    for (int in : {x, res}) all.may_share(total, in);
    all.add("scale", a->scale, rows * 4, true);
  }
  all.add("weight", a->weight, (int64_t)a->channels * 4, false);
  all.add("dweight", a->dweight, (int64_t)a->channels * 4, true);
  if (need) all.add("workspace", ws, need, true);
  DIT_TRY(all.check());
  OnDevice dev;
  if (rows) {
    DIT_TRY(dev.add("x", a->x));
    DIT_TRY(dev.add(res_name, a->residual));
    DIT_TRY(dev.add("total", a->total));
    if (backward) DIT_TRY(dev.add("dy", a->dy));
    DIT_TRY(dev.add("out", a->out));
    DIT_TRY(dev.add("scale", a->scale));
  }
  DIT_TRY(dev.add("weight", a->weight));
  DIT_TRY(dev.add("dweight", a->dweight));
  if (need) DIT_TRY(dev.add("workspace", ws));
  DIT_TRY(dev.enter());
  dit_rms_norm_args c = *a;
  drop_unused(c.x_stride, size);
  drop_unused(c.residual_stride, size);
  drop_unused(c.total_stride, size);
  drop_unused(c.dy_stride, size);
  drop_unused(c.out_stride, size);
  CU_TRY(rms_norm_run(c, backward, static_cast<float*>(ws), stream));
  return DIT_OK;
}

// ---------------------------------------------------------------- gated feed-forward
constexpr int kMaxWidth = 1 << 17;

dit_status check_ffn_shape(const dit_gated_ffn_args* a, bool backward) {
  if (!a) return fail(DIT_ERR_INVALID_ARG, "arguments are NULL");
  if (a->rows < 0 || a->rows > INT32_MAX) return fail(DIT_ERR_SHAPE, "rows must be 0 .. 2^31 - 1");
  if (a->width <= 0 || a->width > kMaxWidth || a->hidden <= 0 || a->hidden > kMaxWidth)
    return fail(DIT_ERR_SHAPE, "width and hidden must be 1 .. 2^17");
  if (a->rows * (a->width > a->hidden ? a->width : a->hidden) > (int64_t)1 << 40)
    return fail(DIT_ERR_SHAPE, "more than 2^40 elements");
  if (a->dtype != DIT_DTYPE_BF16 && a->dtype != DIT_DTYPE_F16)
    return fail(DIT_ERR_INVALID_ARG, "dtype must be bf16 or fp16, is %d", a->dtype);
  if (a->operand_dtype != a->dtype && (backward || a->operand_dtype != DIT_DTYPE_E4M3))
    return fail(DIT_ERR_INVALID_ARG, backward ? "operand_dtype must be dtype" : "operand_dtype must be dtype or e4m3");
  if (a->act != DIT_ACT_SILU && a->act != DIT_ACT_GELU) return fail(DIT_ERR_INVALID_ARG, "act must be SiLU or GELU, is %d", a->act);
  if (a->reserved) return fail(DIT_ERR_INVALID_ARG, "reserved fields must be 0");
  const bool f8 = a->operand_dtype == DIT_DTYPE_E4M3;
  if (f8 ? (!a->x_scale && a->rows) || !a->gate_scale || !a->up_scale : a->x_scale || a->gate_scale || a->up_scale)
    return fail(DIT_ERR_INVALID_ARG, "scales belong to operands in e4m3, which need all three");
  if (!backward && (a->dx || a->dw_gate || a->dw_up || a->dbias_gate || a->dbias_up))
    return fail(DIT_ERR_INVALID_ARG, "gradients belong to the backward call");
  if (backward && (a->bias_gate || a->bias_up)) return fail(DIT_ERR_INVALID_ARG, "the backward call reads no bias");
  if (!a->gate != !a->up && a->rows) return fail(DIT_ERR_INVALID_ARG, "gate and up belong together");
  return DIT_OK;
}

dit_status ffn_call(const dit_gated_ffn_args* a, bool backward, void* ws, int64_t ws_bytes, cudaStream_t stream) {
  clear_last_error();
  DIT_TRY(check_ffn_shape(a, backward));
  const bool some = a->rows > 0;
  const int64_t rows = a->rows, D = a->width, F = a->hidden;
  const int elem = 2, operand = a->operand_dtype == DIT_DTYPE_E4M3 ? 1 : 2;
  const bool dw = a->dw_gate || a->dw_up, db = a->dbias_gate || a->dbias_up;
  if (backward && !a->dx && !dw && !db) return DIT_OK;
  if (!backward && !some) return DIT_OK;
  struct View {
    const char* what;
    const void* p;
    int64_t rows, stride, width;
    int elem;
    bool output, needed;
  };
  // the operands that this call reads, and what it writes
  const View views[] = {
      {"x", a->x, rows, a->x_stride, D, operand, false, some && (!backward || dw)},
      {"w_gate", a->w_gate, F, a->w_gate_stride, D, operand, false, some && (!backward || a->dx)},
      {"w_up", a->w_up, F, a->w_up_stride, D, operand, false, some && (!backward || a->dx)},
      {"gate", a->gate, rows, a->gate_stride, F, elem, !backward, some && (backward || a->gate)},
      {"up", a->up, rows, a->up_stride, F, elem, !backward, some && (backward || a->up)},
      {backward ? "dout" : "out", a->out, rows, a->out_stride, F, elem, !backward, some},
      {"dx", a->dx, rows, a->dx_stride, D, elem, true, some && a->dx},
      {"dw_gate", a->dw_gate, F, a->dw_gate_stride, D, elem, true, a->dw_gate != nullptr},
      {"dw_up", a->dw_up, F, a->dw_up_stride, D, elem, true, a->dw_up != nullptr},
  };
  for (const View& v : views)
    if (v.needed) DIT_TRY(check_view(v.what, v.p, 1, &v.rows, &v.stride, v.width, v.elem, v.output));
  const float* floats[] = {a->x_scale, a->gate_scale, a->up_scale, a->bias_gate, a->bias_up, a->dbias_gate, a->dbias_up};
  const char* names[] = {"x_scale", "gate_scale", "up_scale", "bias_gate", "bias_up", "dbias_gate", "dbias_up"};
  for (const float* p : floats)
    if ((uintptr_t)p % 4) return fail(DIT_ERR_INVALID_ARG, "scales and biases must be aligned to 4 bytes");
  const int64_t need = gated_ffn_workspace(*a, backward);
  DIT_TRY(check_workspace(ws, ws_bytes, need));
  Regions all;
  for (const View& v : views)
    if (v.needed) all.add(v.what, v.p, 1, &v.rows, &v.stride, v.width, v.elem, v.output);
  for (int i = 0; i < 7; ++i) all.add(names[i], floats[i], (i == 0 ? rows : F) * 4, i >= 5);
  if (need) all.add("workspace", ws, need, true);
  DIT_TRY(all.check());
  OnDevice dev;
  for (const View& v : views)
    if (v.needed) DIT_TRY(dev.add(v.what, v.p));
  for (int i = 0; i < 7; ++i) DIT_TRY(dev.add(names[i], floats[i]));
  if (need) DIT_TRY(dev.add("workspace", ws));
  DIT_TRY(dev.enter());
  CU_TRY(gated_ffn_run(*a, backward, ws, stream));
  return DIT_OK;
}

// ---------------------------------------------------------------- gradient norm
dit_status check_grad_tensors(const dit_grad_tensor* t, int64_t n) {
  if (n < 0 || n > INT32_MAX) return fail(DIT_ERR_SHAPE, "the number of tensors must be 0 .. 2^31 - 1");
  if (n && !t) return fail(DIT_ERR_INVALID_ARG, "tensors is NULL");
  int64_t total = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].numel < 0) return fail(DIT_ERR_SHAPE, "tensor %lld has a negative size", (long long)i);
    if (t[i].numel > (int64_t)1 << 44 || (total += t[i].numel) > (int64_t)1 << 44)
      return fail(DIT_ERR_SHAPE, "more than 2^44 elements");
    if (!activation_type(t[i].dtype)) return fail(DIT_ERR_INVALID_ARG, "tensor %lld: unknown dtype %d", (long long)i, t[i].dtype);
    if (t[i].reserved) return fail(DIT_ERR_INVALID_ARG, "reserved fields must be 0");
  }
  return DIT_OK;
}

dit_status grad_norm_call(const dit_grad_tensor* t, int64_t n, float max_norm, float* norm, void* ws, int64_t ws_bytes,
                          cudaStream_t stream) {
  clear_last_error();
  DIT_TRY(check_grad_tensors(t, n));
  if (!(max_norm >= 0.f)) return fail(DIT_ERR_INVALID_ARG, "max_norm must be >= 0");
  if (!norm) return fail(DIT_ERR_INVALID_ARG, "norm is NULL");
  if ((uintptr_t)norm % 4) return fail(DIT_ERR_INVALID_ARG, "norm is not aligned to 4 bytes");
  const bool clip = !isinf(max_norm);
  const int64_t need = grad_norm_workspace(t, n);
  DIT_TRY(check_workspace(ws, ws_bytes, need));
  OnDevice dev;
  // ranges sorted by where they begin: an output has no byte in common with
  // anything else but the gradient that it takes the place of
  struct Range {
    uintptr_t begin, end;
    const char* what;
    bool output;
  };
  std::vector<Range> ranges;
  ranges.reserve(2 * n + 2);
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].numel == 0) continue;
    const int elem = elem_bytes(t[i].dtype);
    if (!t[i].grad) return fail(DIT_ERR_INVALID_ARG, "tensor %lld: grad is NULL", (long long)i);
    if (clip && !t[i].out) return fail(DIT_ERR_INVALID_ARG, "tensor %lld: out is NULL", (long long)i);
    if (!clip && t[i].out) return fail(DIT_ERR_INVALID_ARG, "tensor %lld: out without a finite max_norm", (long long)i);
    if (((uintptr_t)t[i].grad | (uintptr_t)t[i].out) % elem)
      return fail(DIT_ERR_INVALID_ARG, "tensor %lld is not aligned to its type", (long long)i);
    const uintptr_t g = (uintptr_t)t[i].grad, o = (uintptr_t)t[i].out;
    const int64_t bytes = t[i].numel * elem;
    ranges.push_back({g, g + bytes, "grad", o == g});
    if (o && o != g) ranges.push_back({o, o + bytes, "out", true});
  }
  ranges.push_back({(uintptr_t)norm, (uintptr_t)norm + 4, "norm", true});
  ranges.push_back({(uintptr_t)ws, (uintptr_t)ws + need, "workspace", true});
  std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t any_end = 0, out_end = 0;  // furthest end of the ranges before, and of the outputs among them
  for (const Range& r : ranges) {
    if (r.begin < out_end || (r.output && r.begin < any_end))
      return fail(DIT_ERR_INVALID_ARG, "an output overlaps another tensor of the call");
    any_end = std::max(any_end, r.end);
    if (r.output) out_end = std::max(out_end, r.end);
  }
  // The owner of each allocation is looked up once for all ranges that begin in it (a
  // lookup for each of a model's hundreds of tensors took longer than the kernels).
  uintptr_t base = 0;
  size_t size = 0;
  for (const Range& r : ranges) {
    if (r.begin - base < size) continue;
    DIT_TRY(dev.add(r.what, reinterpret_cast<const void*>(r.begin)));
    if (!allocation_of(reinterpret_cast<const void*>(r.begin), &base, &size)) size = 0;
  }
  DIT_TRY(dev.enter());
  CU_TRY(grad_norm_run(t, n, max_norm, norm, ws, stream));
  return DIT_OK;
}

}  // namespace

extern "C" dit_status dit_rms_norm_forward(const dit_rms_norm_args* a, void* stream) {
  return norm_call(a, false, nullptr, 0, static_cast<cudaStream_t>(stream));
}

extern "C" dit_status dit_rms_norm_backward(const dit_rms_norm_args* a, void* ws, int64_t ws_bytes, void* stream) {
  return norm_call(a, true, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int64_t dit_rms_norm_workspace_bytes(const dit_rms_norm_args* a) {
  clear_last_error();
  return check_norm_shape(a, true) == DIT_OK ? rms_norm_workspace(*a) : -1;
}

extern "C" dit_status dit_gated_ffn_forward(const dit_gated_ffn_args* a, void* ws, int64_t ws_bytes, void* stream) {
  return ffn_call(a, false, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" dit_status dit_gated_ffn_backward(const dit_gated_ffn_args* a, void* ws, int64_t ws_bytes, void* stream) {
  return ffn_call(a, true, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int64_t dit_gated_ffn_workspace_bytes(const dit_gated_ffn_args* a, int backward) {
  clear_last_error();
  return check_ffn_shape(a, backward != 0) == DIT_OK ? gated_ffn_workspace(*a, backward != 0) : -1;
}

extern "C" dit_status dit_gated_ffn_synchronize(void* stream) {
  clear_last_error();
  int site = 0;
  CU_TRY(gated_ffn_take_error(&site, static_cast<cudaStream_t>(stream)));
  return site ? fail(DIT_ERR_TIMEOUT, "a kernel of the gated feed-forward abandoned a wait (site %d)", site) : DIT_OK;
}

extern "C" dit_status dit_grad_norm(const dit_grad_tensor* tensors, int64_t n, float max_norm, float* norm, void* ws,
                                    int64_t ws_bytes, void* stream) {
  try {
    return grad_norm_call(tensors, n, max_norm, norm, ws, ws_bytes, static_cast<cudaStream_t>(stream));
  } catch (const std::bad_alloc&) {
    return fail(DIT_ERR_OOM, "no host memory for %lld tensors", (long long)n);
  }
}

extern "C" int64_t dit_grad_norm_workspace_bytes(const dit_grad_tensor* tensors, int64_t n) {
  clear_last_error();
  return check_grad_tensors(tensors, n) == DIT_OK ? grad_norm_workspace(tensors, n) : -1;
}
