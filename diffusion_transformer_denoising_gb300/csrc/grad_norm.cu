// The norm of many tensors together, and their clipping to it.
//
// Mathematics.  norm = sqrt(sum g^2) over every value of every tensor; where it is
// above max_norm, out = g (max_norm / norm).  The squares of a thread's vectors of a
// piece are summed in fp32 while they are in range, in fp64 where a vector's are not
// (values above 1e15 or all below 1e-15), and joined in fp64 in a fixed order.
//
// What bounds it: HBM.  Two passes, since the factor needs every value: the sums of
// the pieces that a block has (always the same ones), then the factor (each block
// adds up the blocks' sums for itself) and the products.  The second pass walks the
// pieces backwards, so it begins with what the first has left in L2.  Measured on one
// GB300: 0.83 G bf16 gradients 235 us = 7.0 TB/s and 500 us = 6.6 TB/s (with a sum for
// each piece, which a block waited for and the second pass read, 468 and 575 us).
#include <math.h>

#include "launch.cuh"
#include "operators.h"
#include "vec.cuh"

namespace dit {

namespace {

// Values a block takes at a time: few where there are few, so that they spread over the card.
constexpr int kPieceSmall = 2048, kPieceLarge = 16384;
constexpr int64_t kFew = (int64_t)1 << 22;
// Tensors of a launch: its parameters hold their descriptions (32764 bytes at most).
// Few are described in fewer bytes, which every launch copies.
constexpr int kTensors = 640, kFewTensors = 32;
constexpr int kGradThreads = 256;
constexpr int kGradBlocks = 152 * 3;  // of a pass over the squares: the sums' order does not depend on the device

template <int N>
struct Tensors {
  const void* grad[N];
  void* out[N];
  int64_t numel[N];
  uint32_t end[N];               // pieces up to and with tensor i, counted over all launches
  int16_t dtype[N];
  int n, piece;                  // tensors; values of a piece
  uint32_t first;                // pieces of the launches before
  uint32_t parts;                // sums of all launches
  uint32_t first_part;
  double* sums;                  // [parts]
  float* norm;
  float max_norm;
  int write_norm;
};
static_assert(sizeof(Tensors<kTensors>) <= 32764, "parameters of a launch");

// The tensor of a piece: the first whose end is above it.
template <int N>
DIT_DEV int tensor_of(const Tensors<N>& t, uint32_t piece) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (t.end[mid] > piece) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Squares of one vector (E values), in fp32 where neither overflow nor underflow
// can matter: the sum of a vector of values that are all below 1e-15 or that has one
// above 1e15 is taken in fp64.  The zeros of a sparse gradient are no such vector.
template <typename T, int E>
DIT_DEV void add_squares(const Raw<T, E>& r, float& fine, double& rest) {
  float f[E], s = 0.f;
  unpack<T, E>(r, f);
#pragma unroll
  for (int j = 0; j < E; ++j) s = fmaf(f[j], f[j], s);
  if (__builtin_expect(s > 1e-30f && s < 1e30f, 1)) {
    fine += s;
    return;
  }
  uint32_t any = 0;
#pragma unroll
  for (int j = 0; j < Raw<T, E>::kWords; ++j) any |= r.w[j];
  if (any == 0) return;
#pragma unroll 1
  for (int j = 0; j < E; ++j) {
    double v = 0.;  // f[j] without an array in local memory
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (k == j) v = (double)f[k];
    rest += v * v;
  }
}

DIT_DEV double block_sum(double v, double* shared) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  v = shared[0];
#pragma unroll
  for (int i = 1; i < kGradThreads / 32; ++i) v += shared[i];
  __syncthreads();
  return v;
}

template <typename T>
DIT_DEV double piece_squares(const T* p, int n) {
  constexpr int E = 16 / sizeof(T), PER = kPieceLarge / (E * kGradThreads);  // vectors a thread
  double rest = 0.;
  float fine = 0.f;
  // values in front of the first 16-byte boundary, then whole vectors, then the rest
  int head = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T);
  head = head < n ? head : n;
  const int vectors = (n - head) / E;
  if (vectors == PER * kGradThreads) {
    Raw<T, E> r[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) r[i] = load_raw<T, E>(p + (i * kGradThreads + threadIdx.x) * E);
#pragma unroll
    for (int i = 0; i < PER; ++i) add_squares<T, E>(r[i], fine, rest);
  } else {
    constexpr int U = 4;  // loads under way
    for (int i = threadIdx.x; i < vectors; i += U * kGradThreads) {
      Raw<T, E> r[U];
#pragma unroll
      for (int k = 0; k < U; ++k) r[k] = i + k * kGradThreads < vectors ? load_raw<T, E>(p + head + (i + k * kGradThreads) * E) : zero_raw<T, E>();
#pragma unroll
      for (int k = 0; k < U; ++k) add_squares<T, E>(r[k], fine, rest);
    }
    const int tail = n - head - vectors * E;
    const int i = (int)threadIdx.x;
    if (i < head + tail) {
      const double v = (double)to_f32(p[i < head ? i : n - tail + i - head]);
      rest += v * v;
    }
  }
  return rest + (double)fine;
}

template <int N>
__global__ void __launch_bounds__(kGradThreads) grad_squares_kernel(const __grid_constant__ Tensors<N> t) {
  __shared__ double shared[kGradThreads / 32];
  const uint32_t last = t.end[t.n - 1];
  double v = 0.;
  for (uint32_t piece = t.first + blockIdx.x; piece < last; piece += gridDim.x) {
    const int i = tensor_of(t, piece);
    const int64_t begin = (int64_t)(piece - (i ? t.end[i - 1] : t.first)) * t.piece;
    const int n = (int)min((int64_t)t.piece, t.numel[i] - begin);
    if (t.dtype[i] == DIT_DTYPE_F32) v += piece_squares(static_cast<const float*>(t.grad[i]) + begin, n);
    else if (t.dtype[i] == DIT_DTYPE_BF16) v += piece_squares(static_cast<const __nv_bfloat16*>(t.grad[i]) + begin, n);
    else v += piece_squares(static_cast<const __half*>(t.grad[i]) + begin, n);
  }
  v = block_sum(v, shared);
  if (threadIdx.x == 0) t.sums[t.first_part + blockIdx.x] = v;
}

template <typename T>
DIT_DEV void scale_piece(const T* p, T* out, int n, float k) {
  constexpr int E = 16 / sizeof(T);
  int head = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T);
  head = head < n ? head : n;
  const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  const int vectors = same ? (n - head) / E : 0;
  if (!same) head = n;
  constexpr int U = 4;  // loads under way before the stores, which may be to the same place
  for (int i = threadIdx.x; i < vectors; i += U * kGradThreads) {
    Raw<T, E> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * kGradThreads < vectors) r[u] = load_raw<T, E>(p + head + (i + u * kGradThreads) * E);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u * kGradThreads >= vectors) continue;
      float f[E];
      unpack<T, E>(r[u], f);
#pragma unroll
      for (int j = 0; j < E; ++j) f[j] *= k;
      store_f32<T, E>(out + head + (i + u * kGradThreads) * E, f);
    }
  }
  for (int i = threadIdx.x; i < n - vectors * E; i += kGradThreads) {
    const int at = i < head ? i : vectors * E + i;
    out[at] = from_f32<T>(to_f32(p[at]) * k);
  }
}

template <int N>
__global__ void __launch_bounds__(kGradThreads) grad_clip_kernel(const __grid_constant__ Tensors<N> t) {
  __shared__ double shared[kGradThreads / 32];
  wait_previous();
  double v = 0.;
  for (uint32_t i = threadIdx.x; i < t.parts; i += kGradThreads) v += t.sums[i];
  v = block_sum(v, shared);
  const float norm = (float)sqrt(v);
  if (t.write_norm && blockIdx.x == 0 && threadIdx.x == 0) *t.norm = norm;
  if (t.n == 0 || !t.out[0]) return;
  // a norm that is NaN or infinite leaves the values as they are
  const bool clip = norm > t.max_norm && norm <= 3.402823466e38f;
  const float k = clip ? (float)((double)t.max_norm / sqrt(v)) : 1.f;
  const uint32_t last = t.end[t.n - 1];
  for (uint32_t j = blockIdx.x; j < last - t.first; j += gridDim.x) {
    const uint32_t piece = last - 1 - j;
    const int i = tensor_of(t, piece);
    if (!clip && t.out[i] == t.grad[i]) continue;
    const int64_t begin = (int64_t)(piece - (i ? t.end[i - 1] : t.first)) * t.piece;
    const int n = (int)min((int64_t)t.piece, t.numel[i] - begin);
    if (t.dtype[i] == DIT_DTYPE_F32) scale_piece(static_cast<const float*>(t.grad[i]) + begin, static_cast<float*>(t.out[i]) + begin, n, k);
    else if (t.dtype[i] == DIT_DTYPE_BF16) scale_piece(static_cast<const __nv_bfloat16*>(t.grad[i]) + begin, static_cast<__nv_bfloat16*>(t.out[i]) + begin, n, k);
    else scale_piece(static_cast<const __half*>(t.grad[i]) + begin, static_cast<__half*>(t.out[i]) + begin, n, k);
  }
}

int piece_size(const dit_grad_tensor* t, int64_t n) {
  int64_t all = 0;
  for (int64_t i = 0; i < n; ++i) all += t[i].numel;
  return all <= kFew ? kPieceSmall : kPieceLarge;
}
int64_t pieces_of(const dit_grad_tensor& t, int piece) { return (t.numel + piece - 1) / piece; }

// One launch's tensors, from tensor i on.
struct Batch {
  int64_t next, pieces;
  int n;
};
Batch batch_of(const dit_grad_tensor* t, int64_t n, int64_t i, int piece) {
  Batch b{i, 0, 0};
  for (; b.next < n && b.n < kTensors; ++b.next)
    if (t[b.next].numel > 0) b.pieces += pieces_of(t[b.next], piece), ++b.n;
  return b;
}
int64_t parts_of(const Batch& b) { return b.pieces < kGradBlocks ? b.pieces : kGradBlocks; }
int64_t all_parts(const dit_grad_tensor* t, int64_t n, int piece) {
  int64_t parts = 0;
  for (int64_t i = 0; i < n;) {
    const Batch b = batch_of(t, n, i, piece);
    parts += parts_of(b);
    i = b.next;
  }
  return parts;
}

}  // namespace

int64_t grad_norm_workspace(const dit_grad_tensor* t, int64_t n) {
  const int64_t parts = all_parts(t, n, piece_size(t, n));
  return (parts > 0 ? parts : 1) * (int64_t)sizeof(double);
}

namespace {

template <int N>
cudaError_t run(const dit_grad_tensor* t, int64_t n, float max_norm, float* norm, void* workspace, cudaStream_t s) {
  bool products = false;
  for (int64_t i = 0; i < n; ++i) products |= t[i].numel > 0 && t[i].out;
  Tensors<N> p;
  p.piece = piece_size(t, n);
  p.parts = (uint32_t)all_parts(t, n, p.piece);
  p.sums = static_cast<double*>(workspace), p.norm = norm, p.max_norm = max_norm;
  // squares of every launch first, then products of every launch
  for (int pass = 0; pass < 2; ++pass) {
    p.first = p.first_part = 0;
    p.write_norm = 1;
    int64_t i = 0;
    do {
      const Batch b = batch_of(t, n, i, p.piece);
      uint32_t end = p.first;
      for (p.n = 0; i < b.next; ++i) {
        if (t[i].numel == 0) continue;
        p.grad[p.n] = t[i].grad, p.out[p.n] = t[i].out, p.numel[p.n] = t[i].numel;
        p.dtype[p.n] = (int16_t)t[i].dtype, p.end[p.n] = end += (uint32_t)pieces_of(t[i], p.piece);
        ++p.n;
      }
      cudaError_t e = cudaSuccess;
      if (pass == 0) {
        if (b.n) e = launch_kernel(grad_squares_kernel<N>, dim3((unsigned)parts_of(b)), dim3(kGradThreads), 0, s, 1, false, p);
      } else {
        const int64_t blocks = !products ? 1 : b.pieces < 152 * 8 ? b.pieces : 152 * 8;
        e = launch_kernel(grad_clip_kernel<N>, dim3((unsigned)(blocks > 0 ? blocks : 1)), dim3(kGradThreads), 0, s, 1, true, p);
      }
      if (e != cudaSuccess) return e;
      p.first = end, p.first_part += (uint32_t)parts_of(b);
      p.write_norm = 0;
    } while (i < n && (pass == 0 || products));
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t grad_norm_run(const dit_grad_tensor* t, int64_t n, float max_norm, float* norm, void* workspace, cudaStream_t s) {
  int64_t some = 0;
  for (int64_t i = 0; i < n; ++i) some += t[i].numel > 0;
  return some <= kFewTensors ? run<kFewTensors>(t, n, max_norm, norm, workspace, s) : run<kTensors>(t, n, max_norm, norm, workspace, s);
}

}  // namespace dit
