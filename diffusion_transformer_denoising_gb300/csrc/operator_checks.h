// Argument checks that the operators' C entries share: views, overlaps, the
// device that owns the tensors, the caller's workspace.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "api_common.h"

namespace dit {

// Sizes and strides stay below this, so that element offsets and byte offsets
// (at most 4 strides x sizes, 4 bytes) cannot pass 63 bits.
constexpr int64_t kMaxExtent = (int64_t)1 << 56;

inline int elem_bytes(int dtype) { return dtype == DIT_DTYPE_F32 ? 4 : 2; }

// A view of n axes (sizes, strides in elements) plus a contiguous last axis:
// strides are non-negative and the last element's offset stays in range; an
// output's elements must not share memory.
inline dit_status check_view(const char* what, const void* p, int n, const int64_t* size, const int64_t* stride, int64_t last,
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
inline dit_status check_in_place(const char* what, const void* in, const int64_t* is, const void* out, const int64_t* os,
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

inline dit_status check_workspace(const void* ws, int64_t bytes, int64_t need) {
  if (need == 0) return DIT_OK;
  if (!ws) return fail(DIT_ERR_INVALID_ARG, "the call needs %lld bytes of workspace", (long long)need);
  if (bytes < need)
    return fail(DIT_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)bytes, (long long)need);
  if ((uintptr_t)ws & 15) return fail(DIT_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  return DIT_OK;
}

}  // namespace dit
