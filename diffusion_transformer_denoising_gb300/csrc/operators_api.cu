// C ABI of the operators beside the model: argument checks on the host, then
// the launch on the device that owns the tensors.
#include <math.h>

#include "operator_checks.h"
#include "operators.h"

using namespace dit;

// the binding packs these structures by hand
static_assert(sizeof(dit_rope_args) == 328 && sizeof(dit_group_norm_args) == 160, "layout of the ABI structures");

namespace {

// ---------------------------------------------------------------- rotation
// Everything but the pointers.
dit_status check_rope_shape(const dit_rope_args* a, bool backward) {
  if (!a) return fail(DIT_ERR_INVALID_ARG, "arguments are NULL");
  if (a->batch < 0 || a->tokens < 0) return fail(DIT_ERR_SHAPE, "negative batch or tokens");
  if (a->batch > INT32_MAX || a->tokens > INT32_MAX || a->batch * a->tokens > INT32_MAX)
    return fail(DIT_ERR_SHAPE, "batch * tokens must be below 2^31");
  if (a->head_dim <= 0 || a->head_dim % 2 || a->head_dim > DIT_ROPE_MAX_HEAD_DIM)
    return fail(DIT_ERR_SHAPE, "head_dim must be even and at most %d", DIT_ROPE_MAX_HEAD_DIM);
  if (a->dtype != DIT_DTYPE_F32 && a->dtype != DIT_DTYPE_BF16 && a->dtype != DIT_DTYPE_F16)
    return fail(DIT_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
  if (a->style != DIT_ROPE_INTERLEAVED && a->style != DIT_ROPE_SPLIT)
    return fail(DIT_ERR_INVALID_ARG, "unknown rotary style %d", a->style);
  if (a->pos_dtype != DIT_POS_I32 && a->pos_dtype != DIT_POS_F32)
    return fail(DIT_ERR_INVALID_ARG, "unknown position dtype %d", a->pos_dtype);
  if (a->n_axes < 1 || a->n_axes > DIT_ROPE_MAX_AXES)
    return fail(DIT_ERR_INVALID_ARG, "n_axes must be 1 .. %d", DIT_ROPE_MAX_AXES);
  int turned = 0;
  for (int i = 0; i < a->n_axes; ++i) {
    if (a->axes[i] < 0 || a->axes[i] % 2 || a->axes[i] > a->head_dim)
      return fail(DIT_ERR_INVALID_ARG, "axes must be even, non-negative and at most head_dim");
    turned += a->axes[i];
  }
  if (turned > a->head_dim) return fail(DIT_ERR_INVALID_ARG, "axes sum %d exceeds head_dim %d", turned, a->head_dim);
  if (!(a->theta >= 1.f) || !isfinite(a->theta)) return fail(DIT_ERR_INVALID_ARG, "theta must be finite and >= 1");
  if (!(a->eps >= 0.f) || !isfinite(a->eps)) return fail(DIT_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (a->reserved || a->q.reserved || a->k.reserved) return fail(DIT_ERR_INVALID_ARG, "reserved fields must be 0");
  if (a->q.heads < 0 || a->k.heads < 0 || a->q.heads > (1 << 16) || a->k.heads > (1 << 16))
    return fail(DIT_ERR_SHAPE, "heads must be 0 .. 65536");
  if (a->q.heads == 0 && a->k.heads == 0) return fail(DIT_ERR_SHAPE, "neither q nor k has heads");
  for (const dit_rope_heads* h : {&a->q, &a->k}) {
    if (h->heads == 0 && (h->weight || h->dweight || h->out))
      return fail(DIT_ERR_INVALID_ARG, "a tensor without heads has pointers");
    if (!backward && h->dweight) return fail(DIT_ERR_INVALID_ARG, "dweight belongs to the backward call");
    if (h->dweight && !h->weight) return fail(DIT_ERR_INVALID_ARG, "dweight without weight");
  }
  if (a->q.dweight && a->q.dweight == a->k.dweight)
    return fail(DIT_ERR_INVALID_ARG, "q and k need a dweight each");
  return DIT_OK;
}

int64_t rope_workspace(const dit_rope_args& a) {
  if ((!a.q.dweight && !a.k.dweight) || a.batch * a.tokens == 0 || rope_one_cluster(a)) return 0;
  return (int64_t)kRopeGradBlocks * a.head_dim * sizeof(float);
}

dit_status rope_call(const dit_rope_args* a, bool backward, void* ws, int64_t ws_bytes, cudaStream_t stream) {
  clear_last_error();
  DIT_TRY(check_rope_shape(a, backward));
  const int64_t rows = a->batch * a->tokens;
  const int elem = elem_bytes(a->dtype);
  OnDevice dev;
  const char* names[2][3] = {{"q.x", "q.dy", "q.out"}, {"k.x", "k.dy", "k.out"}};
  const dit_rope_heads* hs[2] = {&a->q, &a->k};
  if (rows) {
    const int64_t psize[2] = {a->batch, a->tokens};
    DIT_TRY(check_view("pos", a->pos, 2, psize, a->pos_stride, a->n_axes, 4, false));
    for (int i = 0; i < 2; ++i) {
      const dit_rope_heads& h = *hs[i];
      if (!h.heads) continue;
      const int64_t size[3] = {a->batch, a->tokens, h.heads};
      if (!backward || h.weight) {
        DIT_TRY(check_view(names[i][0], h.x, 3, size, h.x_stride, a->head_dim, elem, false));
        DIT_TRY(check_in_place(names[i][0], h.x, h.x_stride, h.out, h.out_stride, size, 3));
      }
      if (backward) {
        DIT_TRY(check_view(names[i][1], h.dy, 3, size, h.dy_stride, a->head_dim, elem, false));
        DIT_TRY(check_in_place(names[i][1], h.dy, h.dy_stride, h.out, h.out_stride, size, 3));
      }
      DIT_TRY(check_view(names[i][2], h.out, 3, size, h.out_stride, a->head_dim, elem, true));
    }
  }
  for (int i = 0; i < 2; ++i)
    if (((uintptr_t)hs[i]->weight | (uintptr_t)hs[i]->dweight) % 4)
      return fail(DIT_ERR_INVALID_ARG, "weights must be aligned to 4 bytes");
  if (!rows && !a->q.dweight && !a->k.dweight) return DIT_OK;
  const int64_t need = backward ? rope_workspace(*a) : 0;
  DIT_TRY(check_workspace(ws, ws_bytes, need));
  Regions all;
  if (rows) {
    const int64_t psize[2] = {a->batch, a->tokens};
    all.add("pos", a->pos, 2, psize, a->pos_stride, a->n_axes, 4, false);
  }
  for (int i = 0; i < 2; ++i) {
    const dit_rope_heads& h = *hs[i];
    const int64_t size[3] = {a->batch, a->tokens, h.heads};
    if (rows && h.heads) {
      const int out = all.add(names[i][2], h.out, 3, size, h.out_stride, a->head_dim, elem, true);
      if (!backward || h.weight)
        all.may_share(out, all.add(names[i][0], h.x, 3, size, h.x_stride, a->head_dim, elem, false));
      if (backward) all.may_share(out, all.add(names[i][1], h.dy, 3, size, h.dy_stride, a->head_dim, elem, false));
    }
    all.add(i ? "k.weight" : "q.weight", h.weight, (int64_t)a->head_dim * 4, false);
    all.add(i ? "k.dweight" : "q.dweight", h.dweight, (int64_t)a->head_dim * 4, true);
  }
  if (need) all.add("workspace", ws, need, true);
  DIT_TRY(all.check());
  if (rows) {
    DIT_TRY(dev.add("pos", a->pos));
    for (int i = 0; i < 2; ++i) {
      const dit_rope_heads& h = *hs[i];
      if (!h.heads) continue;
      if (!backward || h.weight) DIT_TRY(dev.add(names[i][0], h.x));
      if (backward) DIT_TRY(dev.add(names[i][1], h.dy));
      DIT_TRY(dev.add(names[i][2], h.out));
    }
  }
  for (int i = 0; i < 2; ++i) {
    DIT_TRY(dev.add("weight", hs[i]->weight));
    DIT_TRY(dev.add("dweight", hs[i]->dweight));
  }
  if (need) DIT_TRY(dev.add("workspace", ws));
  DIT_TRY(dev.enter());
  dit_rope_args c = *a;
  for (dit_rope_heads* h : {&c.q, &c.k}) {
    const int64_t size[3] = {c.batch, c.tokens, h->heads};
    drop_unused(h->x_stride, size);
    drop_unused(h->dy_stride, size);
    drop_unused(h->out_stride, size);
    if (backward && !h->weight) h->x = nullptr;  // not read
  }
  CU_TRY(rope_run(c, backward, static_cast<float*>(ws), stream));
  return DIT_OK;
}

// ---------------------------------------------------------------- group norm
dit_status check_gn_shape(const dit_group_norm_args* a, bool backward) {
  if (!a) return fail(DIT_ERR_INVALID_ARG, "arguments are NULL");
  if (a->batch < 0 || a->pixels < 0) return fail(DIT_ERR_SHAPE, "negative batch or pixels");
  if (a->channels <= 0 || a->channels > (1 << 20)) return fail(DIT_ERR_SHAPE, "channels must be 1 .. 2^20");
  if (a->groups <= 0 || a->channels % a->groups) return fail(DIT_ERR_SHAPE, "groups must divide channels");
  if (a->pixels > INT32_MAX || a->batch > (1 << 20) || a->batch * a->groups > INT32_MAX)
    return fail(DIT_ERR_SHAPE, "pixels must be below 2^31, batch at most 2^20, batch * groups below 2^31");
  if (a->batch * a->pixels > ((int64_t)1 << 40) / a->channels) return fail(DIT_ERR_SHAPE, "more than 2^40 elements");
  if (a->dtype != DIT_DTYPE_F32 && a->dtype != DIT_DTYPE_BF16 && a->dtype != DIT_DTYPE_F16)
    return fail(DIT_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
  if (a->act != DIT_ACT_NONE && a->act != DIT_ACT_SILU) return fail(DIT_ERR_INVALID_ARG, "unknown act %d", a->act);
  if (!(a->eps >= 0.f) || !isfinite(a->eps)) return fail(DIT_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (a->reserved) return fail(DIT_ERR_INVALID_ARG, "reserved fields must be 0");
  if (!backward && (a->dweight || a->dbias))
    return fail(DIT_ERR_INVALID_ARG, "dweight and dbias belong to the backward call");
  if ((a->dweight && !a->weight) || (a->dbias && !a->bias))
    return fail(DIT_ERR_INVALID_ARG, "dweight needs weight, and dbias bias");
  return DIT_OK;
}

dit_status gn_call(const dit_group_norm_args* a, bool backward, void* ws, int64_t ws_bytes, cudaStream_t stream) {
  clear_last_error();
  DIT_TRY(check_gn_shape(a, backward));
  const int elem = elem_bytes(a->dtype);
  const int64_t size[2] = {a->batch, a->pixels};
  const bool some = a->batch && a->pixels;
  if (some) {
    DIT_TRY(check_view("x", a->x, 2, size, a->x_stride, a->channels, elem, false));
    if (backward) DIT_TRY(check_view("dy", a->dy, 2, size, a->dy_stride, a->channels, elem, false));
    DIT_TRY(check_view("out", a->out, 2, size, a->out_stride, a->channels, elem, true));
    DIT_TRY(check_in_place("x", a->x, a->x_stride, a->out, a->out_stride, size, 2));
    if (backward) DIT_TRY(check_in_place("dy", a->dy, a->dy_stride, a->out, a->out_stride, size, 2));
  }
  if (backward && a->batch && (!a->mean || !a->rstd))
    return fail(DIT_ERR_INVALID_ARG, "the backward call needs the forward's mean and rstd");
  if (a->mean && a->mean == a->rstd) return fail(DIT_ERR_INVALID_ARG, "mean and rstd are the same buffer");
  if (a->dweight && a->dweight == a->dbias) return fail(DIT_ERR_INVALID_ARG, "dweight and dbias are the same buffer");
  if (((uintptr_t)a->weight | (uintptr_t)a->bias | (uintptr_t)a->mean | (uintptr_t)a->rstd | (uintptr_t)a->dweight |
       (uintptr_t)a->dbias) % 4)
    return fail(DIT_ERR_INVALID_ARG, "weights and statistics must be aligned to 4 bytes");
  const int64_t need = group_norm_workspace(*a, backward);
  DIT_TRY(check_workspace(ws, ws_bytes, need));
  Regions all;
  if (some) {
    const int out = all.add("out", a->out, 2, size, a->out_stride, a->channels, elem, true);
    all.may_share(out, all.add("x", a->x, 2, size, a->x_stride, a->channels, elem, false));
    if (backward) all.may_share(out, all.add("dy", a->dy, 2, size, a->dy_stride, a->channels, elem, false));
  }
  const int64_t per_channel = (int64_t)a->channels * 4, per_group = a->batch * a->groups * 4;
  all.add("weight", a->weight, per_channel, false);
  all.add("bias", a->bias, per_channel, false);
  all.add("mean", a->mean, per_group, !backward);
  all.add("rstd", a->rstd, per_group, !backward);
  all.add("dweight", a->dweight, per_channel, true);
  all.add("dbias", a->dbias, per_channel, true);
  if (need) all.add("workspace", ws, need, true);
  DIT_TRY(all.check());
  OnDevice dev;
  if (some) {
    DIT_TRY(dev.add("x", a->x));
    if (backward) DIT_TRY(dev.add("dy", a->dy));
    DIT_TRY(dev.add("out", a->out));
  }
  DIT_TRY(dev.add("weight", a->weight));
  DIT_TRY(dev.add("bias", a->bias));
  DIT_TRY(dev.add("mean", a->mean));
  DIT_TRY(dev.add("rstd", a->rstd));
  DIT_TRY(dev.add("dweight", a->dweight));
  DIT_TRY(dev.add("dbias", a->dbias));
  if (need) DIT_TRY(dev.add("workspace", ws));
  if (dev.owner < 0) return DIT_OK;  // nothing to write
  DIT_TRY(dev.enter());
  dit_group_norm_args c = *a;
  drop_unused(c.x_stride, size);
  drop_unused(c.dy_stride, size);
  drop_unused(c.out_stride, size);
  CU_TRY(group_norm_run(c, backward, static_cast<float*>(ws), stream));
  return DIT_OK;
}

}  // namespace

extern "C" dit_status dit_rope_forward(const dit_rope_args* a, void* stream) {
  return rope_call(a, false, nullptr, 0, static_cast<cudaStream_t>(stream));
}

extern "C" dit_status dit_rope_backward(const dit_rope_args* a, void* ws, int64_t ws_bytes, void* stream) {
  return rope_call(a, true, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int64_t dit_rope_workspace_bytes(const dit_rope_args* a) {
  clear_last_error();
  return check_rope_shape(a, true) == DIT_OK ? rope_workspace(*a) : -1;
}

extern "C" dit_status dit_group_norm_forward(const dit_group_norm_args* a, void* ws, int64_t ws_bytes, void* stream) {
  return gn_call(a, false, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" dit_status dit_group_norm_backward(const dit_group_norm_args* a, void* ws, int64_t ws_bytes, void* stream) {
  return gn_call(a, true, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int64_t dit_group_norm_workspace_bytes(const dit_group_norm_args* a, int backward) {
  clear_last_error();
  return check_gn_shape(a, backward != 0) == DIT_OK ? group_norm_workspace(*a, backward != 0) : -1;
}
