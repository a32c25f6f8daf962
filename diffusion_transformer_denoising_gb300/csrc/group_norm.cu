// Group norm of channels-last activations with an optional SiLU, and its
// gradient.
//
// Mathematics.  Per batch element and group: mean and population variance over
// pixels x channels, xhat = (x - mean) rstd, z = xhat w + b, y = act(z).
// Gradient: dz = dy act'(z); per channel A = sum dz, B = sum dz xhat over the
// pixels; dw = sum_batch B, db = sum_batch A; with the group means
// s1 = mean(w dz), s2 = mean(w dz xhat): dx = rstd (w dz - s1 - xhat s2).
//
// Sums.  A thread owns a run of channels and walks pixels.  It keeps, per
// channel, sums of x - K and (x - K)^2 about a pivot K (its first value, then
// its running mean), and folds them every kFold pixels into (count, mean, M2):
// nothing cancels however large the mean is against the deviation.  Threads,
// blocks and channels of a group are then joined as (count, mean, M2) in a
// fixed order, so results are the same bits every time.
#include "operators.h"
#include "vec.cuh"

namespace dit {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kFold = 32;  // pixels a thread sums before it folds

// sigma(z): ex2 and reciprocal approximations, together below 2^-21 relative.
DIT_DEV float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

struct GnParams {
  const void* x;
  const void* dy;
  void* out;
  int64_t xs[2], ds[2], os[2];
  int64_t batch, pixels;
  int channels, groups, cpg;
  int splits;      // pixel ranges a batch element is cut into
  int slab;        // chunks of V channels a block covers
  int act;
  float eps;
  const float* w;
  const float* b;
  const float* mean;  // [batch, groups], read
  const float* rstd;
  float* mean_out;    // [batch, groups], written by the forward's join
  float* rstd_out;
  float2* part;       // [batch, splits, channels]
  float2* chan;       // [batch, channels]: gradient, (A, B)
  float2* gsum;       // [batch, groups]: gradient, (s1, s2)
  float* dw;
  float* db;
};

DIT_DEV int64_t range_begin(int64_t pixels, int splits, int s) { return pixels * s / splits; }

// The block's channel runs and pixels: thread (row, chunk) takes the run
// `chunk` of the slab and pixels row, row + rows, ... of the block's range.
struct Place {
  int rows, row, c;   // c: first channel of the run
  bool on;
  DIT_DEV Place(const GnParams& P, int V) {
    rows = kThreads / P.slab;
    row = threadIdx.x / P.slab;
    c = (blockIdx.y * P.slab + threadIdx.x % P.slab) * V;
    on = row < rows && c < P.channels;
  }
};

// ---------------------------------------------------------------- forward
// part[b, split, c] = (mean, M2) of the channel over the split's pixels.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_stats_kernel(const __grid_constant__ GnParams P) {
  extern __shared__ float2 sm[];  // [rows][slab * V]
  const Place at(P, V);
  const int64_t b = blockIdx.x / P.splits;
  const int split = blockIdx.x - b * P.splits;
  const int64_t p0 = range_begin(P.pixels, P.splits, split), p1 = range_begin(P.pixels, P.splits, split + 1);
  const T* x = static_cast<const T*>(P.x) + b * P.xs[0] + at.c;
  float K[V], s[V], q[V], M2[V];
  int n = 0, m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) K[i] = s[i] = q[i] = M2[i] = 0.f;
  auto fold = [&] {
    if (!m) return;
    const float im = 1.f / (float)m, f = (float)m / (float)(n + m);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float d = s[i] * im;
      M2[i] += fmaf(-d, s[i], q[i]) + d * d * ((float)n * f);
      K[i] = fmaf(d, f, K[i]);
      s[i] = q[i] = 0.f;
    }
    n += m;
    m = 0;
  };
  if (at.on) {
    for (int64_t p = p0 + at.row; p < p1; p += (int64_t)at.rows * kUnroll) {
      Raw<T, V> r[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (p + u * at.rows < p1) r[u] = load_raw<T, V>(x + (p + u * at.rows) * P.xs[1]);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (p + u * at.rows >= p1) continue;
        float v[V];
        unpack<T, V>(r[u], v);
        if (n + m == 0) {
#pragma unroll
          for (int i = 0; i < V; ++i) K[i] = v[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float d = v[i] - K[i];
          s[i] += d;
          q[i] = fmaf(d, d, q[i]);
        }
        ++m;
      }
      if (m >= kFold) fold();
    }
    fold();
    const int width = P.slab * V, ch = threadIdx.x % P.slab * V;
#pragma unroll
    for (int i = 0; i < V; ++i) sm[at.row * width + ch + i] = make_float2(K[i], M2[i]);
  }
  __syncthreads();
  const int width = P.slab * V, c0 = blockIdx.y * width;
  const int64_t len = p1 - p0;
  for (int ch = threadIdx.x; ch < width && c0 + ch < P.channels; ch += kThreads) {
    // means are joined about the first row's, so a large common mean costs nothing
    float mean = 0.f, M = 0.f;
    const float K = len ? sm[ch].x : 0.f;
    for (int r = 0; r < at.rows; ++r) {
      const float cnt = (float)(len > r ? (len - r + at.rows - 1) / at.rows : 0);
      if (cnt > 0.f) mean = fmaf(cnt, sm[r * width + ch].x - K, mean);
    }
    mean = len ? K + mean / (float)len : 0.f;
    for (int r = 0; r < at.rows; ++r) {
      const float cnt = (float)(len > r ? (len - r + at.rows - 1) / at.rows : 0);
      const float2 e = sm[r * width + ch];
      M += fmaf(cnt * (e.x - mean), e.x - mean, e.y);
    }
    P.part[((int64_t)b * P.splits + split) * P.channels + c0 + ch] = make_float2(mean, M);
  }
}

DIT_DEV float block_sum(float v, float* sm) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) t += sm[i];
  return t;
}

// Joins the partials of one (batch element, group).
__global__ void __launch_bounds__(kThreads) gn_join_kernel(const __grid_constant__ GnParams P) {
  __shared__ float sm[kThreads / 32];
  const int64_t b = blockIdx.x / P.groups;
  const int g = blockIdx.x - b * P.groups;
  const float2* part = P.part + b * P.splits * P.channels + (int64_t)g * P.cpg;
  const int64_t entries = (int64_t)P.splits * P.cpg;
  const float total = (float)P.pixels * (float)P.cpg;
  auto count = [&](int s) { return (float)(range_begin(P.pixels, P.splits, s + 1) - range_begin(P.pixels, P.splits, s)); };
  float v = 0.f;
  const float K = part[0].x;
  for (int64_t i = threadIdx.x; i < entries; i += kThreads) {
    const int s = i / P.cpg, c = i - (int64_t)s * P.cpg;
    v = fmaf(count(s), part[(int64_t)s * P.channels + c].x - K, v);
  }
  const float mean = P.pixels ? K + block_sum(v, sm) / total : 0.f;
  v = 0.f;
  for (int64_t i = threadIdx.x; i < entries; i += kThreads) {
    const int s = i / P.cpg, c = i - (int64_t)s * P.cpg;
    const float2 e = part[(int64_t)s * P.channels + c];
    v += fmaf(count(s) * (e.x - mean), e.x - mean, e.y);
  }
  const float var = P.pixels ? block_sum(v, sm) / total : 0.f;
  if (threadIdx.x == 0) {
    P.mean_out[blockIdx.x] = mean;
    P.rstd_out[blockIdx.x] = 1.f / sqrtf((var < 0.f ? 0.f : var) + P.eps);  // a NaN stays one
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_apply_kernel(const __grid_constant__ GnParams P) {
  const Place at(P, V);
  if (!at.on) return;
  const int64_t b = blockIdx.x / P.splits;
  const int split = blockIdx.x - b * P.splits;
  const int64_t p0 = range_begin(P.pixels, P.splits, split), p1 = range_begin(P.pixels, P.splits, split + 1);
  float mean[V], scale[V], bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t bg = b * P.groups + (at.c + i) / P.cpg;
    mean[i] = P.mean[bg];
    scale[i] = P.rstd[bg] * (P.w ? P.w[at.c + i] : 1.f);
    bias[i] = P.b ? P.b[at.c + i] : 0.f;
  }
  const T* x = static_cast<const T*>(P.x) + b * P.xs[0] + at.c;
  T* y = static_cast<T*>(P.out) + b * P.os[0] + at.c;
  for (int64_t p = p0 + at.row; p < p1; p += (int64_t)at.rows * kUnroll) {
    Raw<T, V> r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (p + u * at.rows < p1) r[u] = load_raw<T, V>(x + (p + u * at.rows) * P.xs[1]);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (p + u * at.rows >= p1) continue;
      float v[V];
      unpack<T, V>(r[u], v);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float z = fmaf(v[i] - mean[i], scale[i], bias[i]);
        v[i] = P.act == DIT_ACT_SILU ? z * sigmoid(z) : z;
      }
      store_f32<T, V>(y + (p + u * at.rows) * P.os[1], v);
    }
  }
}

// ---------------------------------------------------------------- gradient
// dz of one element; xhat as a by-product.
DIT_DEV float dz_of(float x, float dy, float mean, float rstd, float w, float b, int act, float& xhat) {
  xhat = (x - mean) * rstd;
  if (act != DIT_ACT_SILU) return dy;
  const float z = fmaf(xhat, w, b), sg = sigmoid(z);
  return dy * (sg * fmaf(z, 1.f - sg, 1.f));
}

// part[b, split, c] = (sum dz, sum dz xhat) over the split's pixels.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_grad_sums_kernel(const __grid_constant__ GnParams P) {
  extern __shared__ float2 sm[];  // [rows][slab * V]
  const Place at(P, V);
  const int64_t b = blockIdx.x / P.splits;
  const int split = blockIdx.x - b * P.splits;
  const int64_t p0 = range_begin(P.pixels, P.splits, split), p1 = range_begin(P.pixels, P.splits, split + 1);
  const int width = P.slab * V;
  if (at.on) {
    float mean[V], rstd[V], w[V], bias[V], A[V], B[V], ta[V], tb[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t bg = b * P.groups + (at.c + i) / P.cpg;
      mean[i] = P.mean[bg];
      rstd[i] = P.rstd[bg];
      w[i] = P.w ? P.w[at.c + i] : 1.f;
      bias[i] = P.b ? P.b[at.c + i] : 0.f;
      A[i] = B[i] = ta[i] = tb[i] = 0.f;
    }
    const T* x = static_cast<const T*>(P.x) + b * P.xs[0] + at.c;
    const T* dy = static_cast<const T*>(P.dy) + b * P.ds[0] + at.c;
    int m = 0;
    for (int64_t p = p0 + at.row; p < p1; p += (int64_t)at.rows * kUnroll) {
      Raw<T, V> rx[kUnroll], rg[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (p + u * at.rows >= p1) continue;
        rx[u] = load_raw<T, V>(x + (p + u * at.rows) * P.xs[1]);
        rg[u] = load_raw<T, V>(dy + (p + u * at.rows) * P.ds[1]);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (p + u * at.rows >= p1) continue;
        float v[V], g[V];
        unpack<T, V>(rx[u], v);
        unpack<T, V>(rg[u], g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float xh;
          const float dz = dz_of(v[i], g[i], mean[i], rstd[i], w[i], bias[i], P.act, xh);
          ta[i] += dz;
          tb[i] = fmaf(dz, xh, tb[i]);
        }
      }
      m += kUnroll;
      if (m >= kFold) {
        m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) A[i] += ta[i], B[i] += tb[i], ta[i] = tb[i] = 0.f;
      }
    }
    const int ch = threadIdx.x % P.slab * V;
#pragma unroll
    for (int i = 0; i < V; ++i) sm[at.row * width + ch + i] = make_float2(A[i] + ta[i], B[i] + tb[i]);
  }
  __syncthreads();
  const int c0 = blockIdx.y * width;
  for (int ch = threadIdx.x; ch < width && c0 + ch < P.channels; ch += kThreads) {
    float A = 0.f, B = 0.f;
    for (int r = 0; r < at.rows; ++r) A += sm[r * width + ch].x, B += sm[r * width + ch].y;
    P.part[((int64_t)b * P.splits + split) * P.channels + c0 + ch] = make_float2(A, B);
  }
}

// One (batch element, group): per-channel sums over the splits, and the
// group's s1, s2.  Threads (row, column): columns of channels, rows of splits.
__global__ void __launch_bounds__(kThreads) gn_grad_join_kernel(const __grid_constant__ GnParams P, int cols) {
  __shared__ float2 sm[kThreads];
  __shared__ float sums[kThreads / 32];
  const int64_t b = blockIdx.x / P.groups;
  const int g = blockIdx.x - b * P.groups;
  const int rows = kThreads / cols, col = threadIdx.x % cols, row = threadIdx.x / cols;
  const float2* part = P.part + b * P.splits * P.channels + (int64_t)g * P.cpg;
  float s1 = 0.f, s2 = 0.f;
  for (int c0 = 0; c0 < P.cpg; c0 += cols) {
    float A = 0.f, B = 0.f;
    if (c0 + col < P.cpg)
      for (int s = row; s < P.splits; s += rows) {
        const float2 e = part[(int64_t)s * P.channels + c0 + col];
        A += e.x, B += e.y;
      }
    __syncthreads();
    sm[threadIdx.x] = make_float2(A, B);
    __syncthreads();
    if (row == 0 && c0 + col < P.cpg) {
      A = B = 0.f;
      for (int r = 0; r < rows; ++r) A += sm[r * cols + col].x, B += sm[r * cols + col].y;
      const int c = g * P.cpg + c0 + col;
      P.chan[b * P.channels + c] = make_float2(A, B);
      const float w = P.w ? P.w[c] : 1.f;
      s1 = fmaf(w, A, s1), s2 = fmaf(w, B, s2);
    }
  }
  const float total = (float)P.pixels * (float)P.cpg;
  s1 = block_sum(s1, sums);
  s2 = block_sum(s2, sums);
  if (threadIdx.x == 0) P.gsum[blockIdx.x] = P.pixels ? make_float2(s1 / total, s2 / total) : make_float2(0.f, 0.f);
}

// dx; the blocks behind the last pixel range sum the channels over the batch.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_grad_apply_kernel(const __grid_constant__ GnParams P) {
  const int64_t work = P.batch * P.splits;
  if (blockIdx.x >= work) {
    if (blockIdx.y) return;
    const int c = (int)(blockIdx.x - work) * kThreads + threadIdx.x;
    if (c >= P.channels) return;
    float A = 0.f, B = 0.f;
    for (int64_t b = 0; b < P.batch; ++b) A += P.chan[b * P.channels + c].x, B += P.chan[b * P.channels + c].y;
    if (P.db) P.db[c] = A;
    if (P.dw) P.dw[c] = B;
    return;
  }
  const Place at(P, V);
  if (!at.on) return;
  const int64_t b = blockIdx.x / P.splits;
  const int split = blockIdx.x - b * P.splits;
  const int64_t p0 = range_begin(P.pixels, P.splits, split), p1 = range_begin(P.pixels, P.splits, split + 1);
  float mean[V], rstd[V], w[V], bias[V], s1[V], s2[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t bg = b * P.groups + (at.c + i) / P.cpg;
    mean[i] = P.mean[bg];
    rstd[i] = P.rstd[bg];
    w[i] = P.w ? P.w[at.c + i] : 1.f;
    bias[i] = P.b ? P.b[at.c + i] : 0.f;
    const float2 t = P.gsum[bg];
    s1[i] = t.x, s2[i] = t.y;
  }
  const T* x = static_cast<const T*>(P.x) + b * P.xs[0] + at.c;
  const T* dy = static_cast<const T*>(P.dy) + b * P.ds[0] + at.c;
  T* dx = static_cast<T*>(P.out) + b * P.os[0] + at.c;
  for (int64_t p = p0 + at.row; p < p1; p += (int64_t)at.rows * kUnroll) {
    Raw<T, V> rx[kUnroll], rg[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (p + u * at.rows >= p1) continue;
      rx[u] = load_raw<T, V>(x + (p + u * at.rows) * P.xs[1]);
      rg[u] = load_raw<T, V>(dy + (p + u * at.rows) * P.ds[1]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (p + u * at.rows >= p1) continue;
      float v[V], g[V];
      unpack<T, V>(rx[u], v);
      unpack<T, V>(rg[u], g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float xh;
        const float dz = dz_of(v[i], g[i], mean[i], rstd[i], w[i], bias[i], P.act, xh);
        v[i] = rstd[i] * (fmaf(dz, w[i], -s1[i]) - xh * s2[i]);
      }
      store_f32<T, V>(dx + (p + u * at.rows) * P.os[1], v);
    }
  }
}

// ---------------------------------------------------------------- launch
int elem_bytes(int dtype) { return dtype == DIT_DTYPE_F32 ? 4 : 2; }

bool aligned16(const void* p, const int64_t st[2], int elem) {
  return !p || (((uintptr_t)p | (uintptr_t)(st[0] * elem) | (uintptr_t)(st[1] * elem)) & 15) == 0;
}

struct Plan {
  int vec, slab, nslab, splits;
};

Plan plan_of(const dit_group_norm_args& a, int vec) {
  Plan p;
  p.vec = vec;
  const int chunks = a.channels / vec;
  p.nslab = (chunks + kThreads - 1) / kThreads;
  p.slab = (chunks + p.nslab - 1) / p.nslab;
  const int rows = kThreads / p.slab;
  // pixel ranges: about eight blocks an SM in all, at least kUnroll pixels a thread
  int64_t splits = 1216 / (a.batch * p.nslab > 0 ? a.batch * p.nslab : 1);
  const int64_t most = a.pixels / ((int64_t)rows * kUnroll);
  if (splits > most) splits = most;
  p.splits = (int)(splits < 1 ? 1 : splits);
  return p;
}

int vec_of(const dit_group_norm_args& a) {
  const int e = elem_bytes(a.dtype), v = 16 / e;
  const bool ok = a.channels % v == 0 && aligned16(a.x, a.x_stride, e) && aligned16(a.dy, a.dy_stride, e) &&
                  aligned16(a.out, a.out_stride, e);
  return ok ? v : 1;
}

int64_t round256(int64_t n) { return (n + 255) & ~(int64_t)255; }

template <typename T, int V>
cudaError_t run(const dit_group_norm_args& a, const Plan& pl, GnParams P, bool backward, cudaStream_t s) {
  const dim3 grid((unsigned)(a.batch * pl.splits), (unsigned)pl.nslab);
  const size_t sm = (size_t)(kThreads / pl.slab) * pl.slab * V * sizeof(float2);
  const unsigned bg = (unsigned)(a.batch * a.groups);
  if (!backward) {
    gn_stats_kernel<T, V><<<grid, kThreads, sm, s>>>(P);
    gn_join_kernel<<<bg, kThreads, 0, s>>>(P);
    if (a.pixels) gn_apply_kernel<T, V><<<grid, kThreads, 0, s>>>(P);
  } else {
    int cols = 1;
    while (cols < P.cpg && cols < 32) cols *= 2;
    gn_grad_sums_kernel<T, V><<<grid, kThreads, sm, s>>>(P);
    gn_grad_join_kernel<<<bg, kThreads, 0, s>>>(P, cols);
    const unsigned extra = P.dw || P.db ? (a.channels + kThreads - 1) / kThreads : 0;
    gn_grad_apply_kernel<T, V><<<dim3(grid.x + extra, grid.y), kThreads, 0, s>>>(P);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_vec(const dit_group_norm_args& a, const Plan& pl, const GnParams& P, bool backward, cudaStream_t s) {
  if (pl.vec == 1) return run<T, 1>(a, pl, P, backward, s);
  return run<T, 16 / sizeof(T)>(a, pl, P, backward, s);
}

}  // namespace

int64_t group_norm_workspace(const dit_group_norm_args& a, bool backward) {
  if (a.batch == 0) return 0;
  const Plan pl = plan_of(a, vec_of(a));
  const int64_t part = round256(a.batch * pl.splits * (int64_t)a.channels * 8);
  const int64_t bg = round256(a.batch * a.groups * 8);
  return part + bg + (backward ? round256(a.batch * (int64_t)a.channels * 8) : 0);
}

cudaError_t group_norm_run(const dit_group_norm_args& a, bool backward, float* workspace, cudaStream_t stream) {
  GnParams P{};
  const Plan pl = plan_of(a, vec_of(a));
  P.x = a.x;
  P.dy = a.dy;
  P.out = a.out;
  for (int i = 0; i < 2; ++i) P.xs[i] = a.x_stride[i], P.ds[i] = a.dy_stride[i], P.os[i] = a.out_stride[i];
  P.batch = a.batch;
  P.pixels = a.pixels;
  P.channels = a.channels;
  P.groups = a.groups;
  P.cpg = a.channels / a.groups;
  P.splits = pl.splits;
  P.slab = pl.slab;
  P.act = a.act;
  P.eps = a.eps;
  P.w = a.weight;
  P.b = a.bias;
  P.dw = a.dweight;
  P.db = a.dbias;
  if (a.batch == 0) {
    // nothing was summed
    for (float* d : {a.dweight, a.dbias})
      if (backward && d) {
        const cudaError_t e = cudaMemsetAsync(d, 0, (size_t)a.channels * sizeof(float), stream);
        if (e != cudaSuccess) return e;
      }
    return cudaSuccess;
  }
  char* ws = reinterpret_cast<char*>(workspace);
  P.part = reinterpret_cast<float2*>(ws);
  ws += round256(a.batch * pl.splits * (int64_t)a.channels * 8);
  float* bg = reinterpret_cast<float*>(ws);
  ws += round256(a.batch * a.groups * 8);
  if (!backward) {
    P.mean_out = a.mean ? a.mean : bg;
    P.rstd_out = a.rstd ? a.rstd : bg + a.batch * a.groups;
    P.mean = P.mean_out;
    P.rstd = P.rstd_out;
  } else {
    P.mean = a.mean;
    P.rstd = a.rstd;
    P.gsum = reinterpret_cast<float2*>(bg);
    P.chan = reinterpret_cast<float2*>(ws);
  }
  if (a.dtype == DIT_DTYPE_F32) return run_vec<float>(a, pl, P, backward, stream);
  if (a.dtype == DIT_DTYPE_BF16) return run_vec<__nv_bfloat16>(a, pl, P, backward, stream);
  return run_vec<__half>(a, pl, P, backward, stream);
}

}  // namespace dit
