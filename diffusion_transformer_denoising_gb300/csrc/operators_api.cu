// C ABI of the operators beside the model: argument checks on the host, then
// the launch on the device that owns the tensors.
#include <math.h>

#include "api_common.h"
#include "operators.h"

using namespace dit;

// the binding packs these structures by hand
static_assert(sizeof(dit_rope_args) == 328 && sizeof(dit_group_norm_args) == 160, "layout of the ABI structures");

namespace {

// Sizes and strides stay below this, so that element offsets and byte offsets
// (at most 4 strides x sizes, 4 bytes) cannot pass 63 bits.
constexpr int64_t kMaxExtent = (int64_t)1 << 56;

int elem_bytes(int dtype) { return dtype == DIT_DTYPE_F32 ? 4 : 2; }

// A view of n axes (sizes, strides in elements) plus a contiguous last axis:
// strides are non-negative and the last element's offset stays in range; an
// output's elements must not share memory.
dit_status check_view(const char* what, const void* p, int n, const int64_t* size, const int64_t* stride, int64_t last,
                      int elem, bool output) {
  if (!p) return fail(DIT_ERR_INVALID_ARG, "%s is NULL", what);
  if ((uintptr_t)p % elem) return fail(DIT_ERR_INVALID_ARG, "%s is not aligned to its type", what);
  int64_t extent = last;
  for (int i = 0; i < n; ++i) {
    if (stride[i] < 0) return fail(DIT_ERR_SHAPE, "%s has a negative stride", what);
    if (size[i] > 1 && stride[i] > kMaxExtent / size[i]) return fail(DIT_ERR_SHAPE, "%s is too large", what);
    if (size[i] > 1) extent += (size[i] - 1) * stride[i];
    if (extent > kMaxExtent) return fail(DIT_ERR_SHAPE, "%s is too large", what);
  }
  if (!output) return DIT_OK;
  // axes by ascending stride: each must step over all that the smaller ones span
  int order[3] = {0, 1, 2};
  for (int i = 1; i < n; ++i)
    for (int j = i; j > 0 && stride[order[j]] < stride[order[j - 1]]; --j) {
      const int t = order[j];
      order[j] = order[j - 1];
      order[j - 1] = t;
    }
  int64_t span = last;
  for (int i = 0; i < n; ++i) {
    if (size[order[i]] <= 1) continue;
    if (stride[order[i]] < span) return fail(DIT_ERR_SHAPE, "%s: elements of the output share memory", what);
    span += (size[order[i]] - 1) * stride[order[i]];
  }
  return DIT_OK;
}

// An output that starts where an input starts must be the same view.
dit_status check_in_place(const char* what, const void* in, const int64_t* is, const void* out, const int64_t* os,
                          const int64_t* size, int n) {
  if (in != out) return DIT_OK;
  for (int i = 0; i < n; ++i)
    if (size[i] > 1 && is[i] != os[i])
      return fail(DIT_ERR_INVALID_ARG, "%s: an output in place of an input needs the input's strides", what);
  return DIT_OK;
}

// The bytes that a call reads or writes through one pointer: up to three axes
// (strides in bytes) of `last` bytes each.
struct Region {
  const char* what;
  intptr_t p;
  int n;
  int64_t size[3], stride[3], last, span;  // span: from the first byte to the end of the last
};
// Whether two regions have a byte in common.  With x_k the index of a's axis k,
// or minus that of b's, the bytes meet where sum x_k stride_k + (u - v) is the
// distance of the pointers: strides are settled from the largest down, each x_k
// within what the smaller ones can still make up, two values at most where
// strides nest as views of one buffer do.  Views that nest in no way could take
// a long search: it gives up after kSearch steps and finds no overlap then.
struct Overlap {
  static constexpr int kSearch = 4096;
  int n = 0, steps = 0;
  int64_t stride[6], lo[6], hi[6], rest_lo[7], rest_hi[7];

  void axis(int64_t s, int64_t l, int64_t h) {
    for (int k = 0; k < n; ++k)
      if (stride[k] == s) {
        lo[k] += l, hi[k] += h;
        return;
      }
    int k = n++;
    for (; k > 0 && stride[k - 1] < s; --k) stride[k] = stride[k - 1], lo[k] = lo[k - 1], hi[k] = hi[k - 1];
    stride[k] = s, lo[k] = l, hi[k] = h;
  }
  bool meet(int k, int64_t d) {
    if (k == n) return true;  // rest_lo[n] <= d <= rest_hi[n]
    if (++steps > kSearch) return false;
    const int64_t s = stride[k], from = d - rest_hi[k + 1], to = d - rest_lo[k + 1];
    int64_t x = from / s, last = to / s;
    if (x * s < from) ++x;
    if (last * s > to) --last;
    if (x < lo[k]) x = lo[k];
    if (last > hi[k]) last = hi[k];
    for (; x <= last && steps <= kSearch; ++x)
      if (meet(k + 1, d - x * s)) return true;
    return false;
  }
  bool operator()(const Region& a, const Region& b) {
    for (int i = 0; i < a.n; ++i) axis(a.stride[i], 0, a.size[i] - 1);
    for (int i = 0; i < b.n; ++i) axis(b.stride[i], -(b.size[i] - 1), 0);
    rest_lo[n] = 1 - b.last, rest_hi[n] = a.last - 1;
    for (int k = n - 1; k >= 0; --k) rest_lo[k] = rest_lo[k + 1] + lo[k] * stride[k], rest_hi[k] = rest_hi[k + 1] + hi[k] * stride[k];
    const int64_t d = b.p - a.p;
    return d >= rest_lo[0] && d <= rest_hi[0] && meet(0, d);
  }
};

// The regions of a call.  An output has no byte in common with anything else of
// the call, but that an activation output may be (and by check_in_place then is)
// the view of an input that it is computed from.
struct Regions {
  Region r[12];
  int n = 0;
  uint32_t written = 0, in_place[12] = {};  // masks of regions
  // a view of n axes (sizes, strides in elements) plus a contiguous last axis; NULL and empty ones are none
  int add(const char* what, const void* p, int axes, const int64_t* size, const int64_t* stride, int64_t last, int elem,
          bool output) {
    if (!p || last == 0) return -1;
    Region& v = r[n];
    v.what = what;
    v.p = reinterpret_cast<intptr_t>(p);
    v.n = 0;
    v.last = v.span = last * elem;
    for (int i = 0; i < axes; ++i) {
      if (size[i] <= 1 || stride[i] == 0) continue;  // adds no bytes
      v.size[v.n] = size[i];
      v.stride[v.n++] = stride[i] * elem;
      v.span += (size[i] - 1) * stride[i] * elem;
    }
    if (output) written |= 1u << n;
    return n++;
  }
  int add(const char* what, const void* p, int64_t bytes, bool output) { return add(what, p, 0, nullptr, nullptr, bytes, 1, output); }
  void may_share(int out, int in) {
    if (out >= 0 && in >= 0 && r[out].p == r[in].p) in_place[out] |= 1u << in;
  }
  dit_status check() const {
    for (int i = 0; i < n; ++i) {
      if (!(written >> i & 1)) continue;
      const uint32_t skip = (written & ((2u << i) - 1)) | in_place[i];  // itself, and pairs looked at already
      for (int j = 0; j < n; ++j) {
        if (skip >> j & 1 || r[i].p >= r[j].p + r[j].span || r[j].p >= r[i].p + r[i].span) continue;
        if (Overlap()(r[i], r[j])) return fail(DIT_ERR_INVALID_ARG, "%s overlaps %s", r[i].what, r[j].what);
      }
    }
    return DIT_OK;
  }
};

// Strides of axes with one element say nothing, whatever a view gives for them.
template <int N>
void drop_unused(int64_t (&stride)[N], const int64_t* size) {
  for (int i = 0; i < N; ++i)
    if (size[i] <= 1) stride[i] = 0;
}

// The device that owns the tensors; made current for the call, and the
// caller's put back afterwards.
struct OnDevice {
  int before = -1, owner = -1;
  dit_status add(const char* what, const void* p) {
    if (!p) return DIT_OK;
    cudaPointerAttributes at;
    const cudaError_t e = cudaPointerGetAttributes(&at, p);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return fail(DIT_ERR_CUDA, "cudaPointerGetAttributes failed for %s: %s", what, cudaGetErrorString(e));
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
      return fail(DIT_ERR_INVALID_ARG, "%s is not device memory", what);
    if (owner >= 0 && at.device != owner)
      return fail(DIT_ERR_INVALID_ARG, "%s is on device %d, another tensor on device %d", what, at.device, owner);
    owner = at.device;
    return DIT_OK;
  }
  dit_status enter() {
    CU_TRY(cudaGetDevice(&before));
    if (owner >= 0 && owner != before) CU_TRY(cudaSetDevice(owner));
    return DIT_OK;
  }
  ~OnDevice() {
    if (before >= 0 && owner >= 0 && owner != before) cudaSetDevice(before);
  }
};

dit_status check_workspace(const void* ws, int64_t bytes, int64_t need) {
  if (need == 0) return DIT_OK;
  if (!ws) return fail(DIT_ERR_INVALID_ARG, "the call needs %lld bytes of workspace", (long long)need);
  if (bytes < need)
    return fail(DIT_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)bytes, (long long)need);
  if ((uintptr_t)ws & 15) return fail(DIT_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  return DIT_OK;
}

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
