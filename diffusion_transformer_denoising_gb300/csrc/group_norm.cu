// Group norm of channels-last activations with an optional SiLU, and its
// gradient.
//
// Mathematics.  Per batch element and group: mean and population variance over
// pixels x channels, xhat = (x - mean) rstd, z = xhat w + b, y = act(z).
// Gradient: dz = dy act'(z); per channel A = sum dz, B = sum dz xhat over the
// pixels; dw = sum_batch B, db = sum_batch A; with the group means
// s1 = mean(w dz), s2 = mean(w dz xhat): dx = rstd (w dz - s1 - xhat s2).
//
// Sums.  A thread owns a run of V channels and walks pixels.  It keeps, per
// channel, sums of x - K and (x - K)^2 about a pivot K (its first value, then
// its running mean), and folds them every 32 pixels into (count, mean, M2):
// nothing cancels however large the mean is against the deviation.  Threads,
// channels of a group and blocks are then joined as (count, mean, M2) in a
// fixed order, so results are the same bits every time.
//
// What bounds it: HBM and the second look at x.  Two forms:
//   - whole groups of a batch element that fit a cluster's shared memory: one
//     launch.  A block loads its pixels once, into shared memory, the cluster
//     joins the groups' sums through distributed shared memory, and the block
//     writes its pixels out of shared memory: one read, one write.
//   - otherwise three launches chained by programmatic dependence: sums per
//     (pixel range, group), a join per (batch element, group), and a pass that
//     walks the pixel ranges backwards, so that what the sums read last is
//     still in L2.
#include <stdio.h>
#include <stdlib.h>
#include "launch.cuh"
#include "operators.h"
#include "vec.cuh"

namespace dit {

namespace {

constexpr int kThreads = 256;
constexpr int kSumUnroll = 4;    // pixels in flight a thread: forward
constexpr int kPassUnroll = 4;
constexpr int kGradUnroll = 2;   // gradient: of both tensors
constexpr int kFold = 32;        // pixels a thread sums before it folds

struct GnParams {
  const void* x;
  const void* dy;
  void* out;
  int64_t xs[2], ds[2], os[2];
  int64_t batch, pixels;
  int channels, groups, cpg;
  int splits;      // pixel ranges a batch element is cut into
  int passes;      // the same for the pass that writes
  int slab;        // runs of V channels a block covers
  int unit;        // channels of one partial: cpg where slabs hold whole groups, else 1
  int act;
  float eps;
  const float* w;
  const float* b;
  const float* mean;  // [batch, groups], read
  const float* rstd;
  float* mean_out;    // [batch, groups], written, or NULL (cluster form)
  float* rstd_out;
  float2* part;       // forward [batch, splits, channels / unit], gradient [batch, splits, channels]
  float2* chan;       // [batch, channels]: gradient, (A, B)
  float2* gsum;       // [batch, groups]: gradient, (s1, s2)
  float* dw;
  float* db;
};

// ---------------------------------------------------------------- arithmetic
// V values, as fma.rn.f32x2 pairs where V is even.
template <int V, class F2, class F1>
DIT_DEV void each(F2 f2, F1 f1) {
  if constexpr (V % 2) {
#pragma unroll
    for (int i = 0; i < V; ++i) f1(i);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) f2(i);
  }
}
template <int V>
DIT_DEV void v_add(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
  each<V>([&](int i) { const float2 r = fadd2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1])); d[i] = r.x, d[i + 1] = r.y; },
          [&](int i) { d[i] = a[i] + b[i]; });
}
template <int V>
DIT_DEV void v_sub(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
  each<V>([&](int i) { const float2 r = fadd2(make_float2(a[i], a[i + 1]), make_float2(-b[i], -b[i + 1])); d[i] = r.x, d[i + 1] = r.y; },
          [&](int i) { d[i] = a[i] - b[i]; });
}
template <int V>
DIT_DEV void v_mul(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
  each<V>([&](int i) { const float2 r = fmul2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1])); d[i] = r.x, d[i + 1] = r.y; },
          [&](int i) { d[i] = a[i] * b[i]; });
}
template <int V>
DIT_DEV void v_fma(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
  each<V>([&](int i) {
            const float2 r = ffma2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(c[i], c[i + 1]));
            d[i] = r.x, d[i + 1] = r.y;
          },
          [&](int i) { d[i] = fmaf(a[i], b[i], c[i]); });
}
template <int V>
DIT_DEV void v_set(float (&d)[V], float v) {
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = v;
}

DIT_DEV float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// sigma(z) = 1 / (1 + 2^(-z log2 e)): an ex2 and a reciprocal approximation,
// together below 2^-21 relative.
template <int V>
DIT_DEV void v_sigmoid(float (&d)[V], const float (&z)[V]) {
  float k[V], one[V], t[V];
  v_set(k, -1.4426950408889634f);
  v_set(one, 1.f);
  v_mul(t, z, k);
#pragma unroll
  for (int i = 0; i < V; ++i) t[i] = ex2_approx(t[i]);
  v_add(t, t, one);
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = rcp_approx(t[i]);
}

DIT_DEV int64_t range_begin(int64_t pixels, int splits, int s) { return pixels * s / splits; }

// ---------------------------------------------------------------- blocks
// Thread (row, run) takes run `run` of the slab and pixels row, row + rows,
// ... of the block's range [p0, p1).
struct Place {
  int rows, row, run, c, count;
  int64_t p;
  bool on;
  DIT_DEV Place(const GnParams& P, int V, int slab_index, int64_t p0, int64_t p1) {
    rows = kThreads / P.slab;
    row = threadIdx.x / P.slab;
    run = threadIdx.x - row * P.slab;
    c = (slab_index * P.slab + run) * V;
    on = row < rows && c < P.channels;
    p = p0 + row;
    count = on && p < p1 ? (int)((p1 - p + rows - 1) / rows) : 0;
  }
};

// Calls body(i, raw...) for pixels 0 .. count - 1 of a thread, U loads of each
// tensor ahead.
template <typename T, int V, int U, class Body>
DIT_DEV void walk(const T* x, int64_t step, int count, Body body) {
  int i = 0;
  for (; i + U <= count; i += U) {
    Raw<T, V> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = load_raw<T, V>(x + u * step);
    x += U * step;
#pragma unroll
    for (int u = 0; u < U; ++u) body(i + u, r[u]);
  }
  Raw<T, V> r[U - 1];
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (i + u < count) r[u] = load_raw<T, V>(x + u * step);
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (i + u < count) body(i + u, r[u]);
}
template <typename T, int V, int U, class Body>
DIT_DEV void walk2(const T* x, int64_t xstep, const T* g, int64_t gstep, int count, Body body) {
  int i = 0;
  for (; i + U <= count; i += U) {
    Raw<T, V> r[U], q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = load_raw<T, V>(x + u * xstep), q[u] = load_raw<T, V>(g + u * gstep);
    x += U * xstep;
    g += U * gstep;
#pragma unroll
    for (int u = 0; u < U; ++u) body(i + u, r[u], q[u]);
  }
  Raw<T, V> r[U - 1], q[U - 1];
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (i + u < count) r[u] = load_raw<T, V>(x + u * xstep), q[u] = load_raw<T, V>(g + u * gstep);
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (i + u < count) body(i + u, r[u], q[u]);
}

// A thread's mean and M2 per channel.
template <int V>
struct Moments {
  float K[V], s[V], q[V], M2[V];
  int n, m;
  DIT_DEV Moments() : n(0), m(0) { v_set(K, 0.f), v_set(s, 0.f), v_set(q, 0.f), v_set(M2, 0.f); }
  DIT_DEV void add(const float (&v)[V]) {
    if (n + m == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) K[i] = v[i];
    }
    float d[V];
    v_sub(d, v, K);
    v_add(s, s, d);
    v_fma(q, d, d, q);
    if (++m == kFold) fold();
  }
  DIT_DEV void fold() {
    if (!m) return;
    const float im = 1.f / (float)m, f = (float)m / (float)(n + m), g = (float)n * f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float d = s[i] * im;
      M2[i] += fmaf(-d, s[i], q[i]) + d * d * g;
      K[i] = fmaf(d, f, K[i]);
      s[i] = q[i] = 0.f;
    }
    n += m;
    m = 0;
  }
};

template <typename T, int V>
DIT_DEV void store_raw(T* p, const Raw<T, V>& r) {
  constexpr int B = Raw<T, V>::kBytes;
  if constexpr (B >= 16) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
  } else if constexpr (B == 4) {
    *reinterpret_cast<uint32_t*>(p) = r.w[0];
  } else {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)r.w[0];
  }
}

// Per-channel pairs of a block's rows in shared memory, [rows][V][slab]: a
// warp's accesses fall on consecutive words.
DIT_DEV int pair_at(int V, int slab, int c) { return c % V * slab + c / V; }  // channel c of row 0

// Joins the rows' (count, mean, M2) of every channel into row 0 of sm,
// halving the rows; cnt[rows] is scratch.
template <int V>
DIT_DEV void join_rows(const Place& at, Moments<V>& A, float2* sm, float* cnt, int slab) {
  auto put = [&](int row) { return sm + row * V * slab + at.run; };
  float n = (float)at.count;
  if (at.row < at.rows) {
#pragma unroll
    for (int i = 0; i < V; ++i) put(at.row)[i * slab] = make_float2(A.K[i], A.M2[i]);
    if (at.run == 0) cnt[at.row] = n;
  }
  for (int rows = at.rows; rows > 1;) {
    const int h = (rows + 1) / 2;
    __syncthreads();
    if (at.row + h < rows) {
      const float nb = cnt[at.row + h];
      if (nb > 0.f) {
        const float f = nb / (n + nb), g = n * f;
        n += nb;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 o = put(at.row + h)[i * slab];
          const float d = o.x - A.K[i];
          A.K[i] = fmaf(d, f, A.K[i]);
          A.M2[i] += fmaf(d * d, g, o.y);
          put(at.row)[i * slab] = make_float2(A.K[i], A.M2[i]);
        }
        if (at.run == 0) cnt[at.row] = n;
      }
    }
    rows = h;
  }
  __syncthreads();
}

// The same for plain sums.
template <int V>
DIT_DEV void add_rows(const Place& at, float (&A)[V], float (&B)[V], float2* sm, int slab) {
  auto put = [&](int row) { return sm + row * V * slab + at.run; };
  if (at.row < at.rows) {
#pragma unroll
    for (int i = 0; i < V; ++i) put(at.row)[i * slab] = make_float2(A[i], B[i]);
  }
  for (int rows = at.rows; rows > 1;) {
    const int h = (rows + 1) / 2;
    __syncthreads();
    if (at.row + h < rows) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 o = put(at.row + h)[i * slab];
        A[i] += o.x, B[i] += o.y;
        put(at.row)[i * slab] = make_float2(A[i], B[i]);
      }
    }
    rows = h;
  }
  __syncthreads();
}

DIT_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Joins the channels of every group of the slab, each of `len` pixels, from
// row 0 of sm; out(g, mean, M2).  A thread a group of few channels, a warp one
// of many.
template <int V, class Out>
DIT_DEV void join_channels(const float2* sm, int slab, int groups, int cpg, float len, Out out) {
  if (cpg <= 8) {
    for (int g = threadIdx.x; g < groups; g += kThreads) {
      auto e = [&](int c) { return sm[pair_at(V, slab, g * cpg + c)]; };
      const float K = e(0).x;
      float mean = 0.f, M = 0.f;
      for (int c = 1; c < cpg; ++c) mean += e(c).x - K;
      mean = K + mean / (float)cpg;
      for (int c = 0; c < cpg; ++c) M += fmaf(len * (e(c).x - mean), e(c).x - mean, e(c).y);
      out(g, mean, M);
    }
  } else {
    const int lane = threadIdx.x & 31;
    for (int g = threadIdx.x >> 5; g < groups; g += kThreads / 32) {
      auto e = [&](int c) { return sm[pair_at(V, slab, g * cpg + c)]; };
      const float K = e(0).x;
      float mean = 0.f, M = 0.f;
      for (int c = lane; c < cpg; c += 32) mean += e(c).x - K;
      mean = K + warp_sum(mean) / (float)cpg;
      for (int c = lane; c < cpg; c += 32) M += fmaf(len * (e(c).x - mean), e(c).x - mean, e(c).y);
      M = warp_sum(M);
      if (lane == 0) out(g, mean, M);
    }
  }
}

DIT_DEV float rstd_of(float var, float eps) {
  return 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);  // a NaN stays one
}

// y of one run: z = (x - mean) (rstd w) + b, then the activation.
template <int V>
struct Affine {
  float mean[V], scale[V], bias[V];
  DIT_DEV void weights(const GnParams& P, int c) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      scale[i] = P.w ? P.w[c + i] : 1.f;
      bias[i] = P.b ? P.b[c + i] : 0.f;
    }
  }
  // statistics of channel c's group: mean(g), rstd(g)
  template <class S>
  DIT_DEV void statistics(int c, int cpg, S stat) {
    int g = c / cpg, left = cpg - (c - g * cpg);
    float2 t = stat(g);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (left == 0) t = stat(++g), left = cpg;
      --left;
      mean[i] = t.x;
      scale[i] *= t.y;
    }
  }
  DIT_DEV void z(float (&v)[V]) const {
    v_sub(v, v, mean);
    v_fma(v, v, scale, bias);
  }
};
template <int V>
DIT_DEV void activate(float (&v)[V], int act) {
  if (act == DIT_ACT_SILU) {
    float s[V];
    v_sigmoid(s, v);
    v_mul(v, v, s);
  }
}

// ---------------------------------------------------------------- forward, three launches
// part[b, split, unit] = (mean, M2) of the unit's channels over the split.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 3) gn_sums_kernel(const __grid_constant__ GnParams P) {
  extern __shared__ float2 sm[];  // [rows][slab * V], then cnt[rows]
  start_next();
  const int64_t b = blockIdx.x / P.splits;
  const int split = blockIdx.x - b * P.splits;
  const int64_t p0 = range_begin(P.pixels, P.splits, split), p1 = range_begin(P.pixels, P.splits, split + 1);
  const Place at(P, V, blockIdx.y, p0, p1);
  Moments<V> A;
  walk<T, V, kSumUnroll>(static_cast<const T*>(P.x) + b * P.xs[0] + at.p * P.xs[1] + at.c, at.rows * P.xs[1], at.count,
                         [&](int, const Raw<T, V>& r) {
                           float v[V];
                           unpack<T, V>(r, v);
                           A.add(v);
                         });
  A.fold();
  const int width = P.slab * V, c0 = blockIdx.y * width;
  join_rows<V>(at, A, sm, reinterpret_cast<float*>(sm + at.rows * width), P.slab);
  const int here = min(width, P.channels - c0);
  float2* part = P.part + ((b * P.splits + split) * P.channels + c0) / P.unit;
  if (P.unit == 1) {
    for (int c = threadIdx.x; c < here; c += kThreads) part[c] = sm[pair_at(V, P.slab, c)];
  } else {
    join_channels<V>(sm, P.slab, here / P.cpg, P.cpg, (float)(p1 - p0),
                     [&](int g, float mean, float M) { part[g] = make_float2(mean, M); });
  }
}

// (count, mean, M2) of two sets joined into the first.
struct Joint {
  float n, mean, M;
  DIT_DEV void take(float on, float omean, float oM) {
    if (on == 0.f) return;
    if (n == 0.f) {
      n = on, mean = omean, M = oM;
      return;
    }
    const float f = on / (n + on), d = omean - mean;
    M += fmaf(d * d, n * f, oM);
    mean = fmaf(d, f, mean);
    n += on;
  }
};

// Joins the partials of one (batch element, group).
constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads) gn_join_kernel(const __grid_constant__ GnParams P) {
  __shared__ Joint sm[kJoinThreads / 32];
  start_next();
  const int64_t b = blockIdx.x / P.groups;
  const int g = blockIdx.x - b * P.groups;
  const int per = P.cpg / P.unit, stride = P.channels / P.unit;
  const float2* part = P.part + b * P.splits * stride + (int64_t)g * per;
  const int64_t entries = (int64_t)P.splits * per;
  Joint J{0.f, 0.f, 0.f};
  wait_previous();
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < entries; i += kJoinThreads) {
    const int s = per == 1 ? (int)i : (int)(i / per);
    const float2 e = part[(int64_t)s * stride + (i - (int64_t)s * per)];
    J.take((float)(range_begin(P.pixels, P.splits, s + 1) - range_begin(P.pixels, P.splits, s)) * (float)P.unit, e.x, e.y);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float n = __shfl_down_sync(0xFFFFFFFFu, J.n, o), m = __shfl_down_sync(0xFFFFFFFFu, J.mean, o);
    J.take(n, m, __shfl_down_sync(0xFFFFFFFFu, J.M, o));
  }
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = J;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < kJoinThreads / 32; ++i) J.take(sm[i].n, sm[i].mean, sm[i].M);
    P.mean_out[blockIdx.x] = J.mean;
    P.rstd_out[blockIdx.x] = rstd_of(J.n > 0.f ? J.M / J.n : 0.f, P.eps);
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 4) gn_apply_kernel(const __grid_constant__ GnParams P) {
  // backwards: the ranges that the sums read last first
  const int64_t at_block = gridDim.x - 1 - blockIdx.x;
  const int64_t b = at_block / P.passes;
  const int split = at_block - b * P.passes;
  const int64_t p0 = range_begin(P.pixels, P.passes, split), p1 = range_begin(P.pixels, P.passes, split + 1);
  const Place at(P, V, blockIdx.y, p0, p1);
  Affine<V> f;
  if (at.on) f.weights(P, at.c);
  wait_previous();
  if (!at.on) return;
  f.statistics(at.c, P.cpg, [&](int g) { return make_float2(P.mean[b * P.groups + g], P.rstd[b * P.groups + g]); });
  T* y = static_cast<T*>(P.out) + b * P.os[0] + at.p * P.os[1] + at.c;
  const int64_t ystep = at.rows * P.os[1];
  walk<T, V, kPassUnroll>(static_cast<const T*>(P.x) + b * P.xs[0] + at.p * P.xs[1] + at.c, at.rows * P.xs[1], at.count,
                          [&](int, const Raw<T, V>& r) {
                            float v[V];
                            unpack<T, V>(r, v);
                            f.z(v);
                            activate(v, P.act);
                            store_f32<T, V>(y, v);
                            y += ystep;
                          });
}

// ---------------------------------------------------------------- forward, one launch
DIT_DEV float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
DIT_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
DIT_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
constexpr int kMaxCluster = 8;

// A cluster of `splits` blocks takes one slab (whole groups) of one batch
// element; each block keeps its pixels in shared memory, every thread reading
// back only what it wrote itself.
// Shared memory: sums [rows][slab * V] float2, cnt[rows] padded to 256 floats,
// own [groups of the slab] float2 (read by the cluster), stat likewise, data.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 2) gn_cluster_kernel(const __grid_constant__ GnParams P) {
  extern __shared__ float4 raw_sm[];
  const int width = P.slab * V, rows = kThreads / P.slab, slab_groups = width / P.cpg;
  float2* sm = reinterpret_cast<float2*>(raw_sm);
  float* cnt = reinterpret_cast<float*>(sm + rows * width);
  float2* own = reinterpret_cast<float2*>(cnt + kThreads);
  float2* stat = own + slab_groups;
  T* data = reinterpret_cast<T*>(raw_sm) +
            ((reinterpret_cast<char*>(stat + slab_groups) - reinterpret_cast<char*>(raw_sm) + 15) / 16 * 16) / sizeof(T);

  const int rank = blockIdx.x % P.splits;
  const int64_t b = blockIdx.x / P.splits;
  const int64_t p0 = range_begin(P.pixels, P.splits, rank), p1 = range_begin(P.pixels, P.splits, rank + 1);
  const Place at(P, V, blockIdx.y, p0, p1);
  T* mine = data + threadIdx.x * V;
  Moments<V> A;
  walk<T, V, kSumUnroll>(static_cast<const T*>(P.x) + b * P.xs[0] + at.p * P.xs[1] + at.c, at.rows * P.xs[1], at.count,
                         [&](int i, const Raw<T, V>& r) {
                           float v[V];
                           store_raw<T, V>(mine + i * (kThreads * V), r);
                           unpack<T, V>(r, v);
                           A.add(v);
                         });
  A.fold();
  Affine<V> f;
  if (at.on) f.weights(P, at.c);
  join_rows<V>(at, A, sm, cnt, P.slab);
  const int c0 = blockIdx.y * width, groups = min(width, P.channels - c0) / P.cpg, g0 = c0 / P.cpg;
  join_channels<V>(sm, P.slab, groups, P.cpg, (float)(p1 - p0),
                   [&](int g, float mean, float M) { own[g] = make_float2(mean, M); });
  cluster_arrive();
  cluster_wait();
  const float total = (float)P.pixels * (float)P.cpg;
  for (int g = threadIdx.x; g < groups; g += kThreads) {
    float2 e[kMaxCluster];
    float n[kMaxCluster], mean = 0.f, M = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      e[r] = make_float2(0.f, 0.f);
      n[r] = 0.f;
      if (r >= P.splits) continue;
      e[r] = ld_cluster_f2(cluster_map(own + g, r));
      n[r] = (float)(range_begin(P.pixels, P.splits, r + 1) - range_begin(P.pixels, P.splits, r)) * (float)P.cpg;
    }
    // the last block always has pixels
    float K = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) K = r == P.splits - 1 ? e[r].x : K;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (n[r] > 0.f) mean = fmaf(n[r], e[r].x - K, mean);
    mean = K + mean / total;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (n[r] > 0.f) M += fmaf(n[r] * (e[r].x - mean), e[r].x - mean, e[r].y);
    const float rstd = rstd_of(M / total, P.eps);
    stat[g] = make_float2(mean, rstd);
    if (rank == 0) {
      if (P.mean_out) P.mean_out[b * P.groups + g0 + g] = mean;
      if (P.rstd_out) P.rstd_out[b * P.groups + g0 + g] = rstd;
    }
  }
  __syncthreads();
  cluster_arrive();  // this block has read its peers' memory
  if (at.on) {
    f.statistics(at.c, P.cpg, [&](int g) { return stat[g - g0]; });
    T* y = static_cast<T*>(P.out) + b * P.os[0] + at.p * P.os[1] + at.c;
    const int64_t ystep = at.rows * P.os[1];
#pragma unroll 4
    for (int i = 0; i < at.count; ++i) {
      float v[V];
      unpack<T, V>(load_raw<T, V>(mine + i * (kThreads * V)), v);
      f.z(v);
      activate(v, P.act);
      store_f32<T, V>(y, v);
      y += ystep;
    }
  }
  cluster_wait();  // a block's memory stays until every peer has read it
}

// ---------------------------------------------------------------- gradient
// dz of one run and xm = x - mean; B sums dz xm, and takes its rstd at the end.
template <int V>
DIT_DEV void dz_of(const Affine<V>& f, const float (&x)[V], const float (&dy)[V], int act, float (&xm)[V], float (&dz)[V]) {
  v_sub(xm, x, f.mean);
  if (act == DIT_ACT_SILU) {
    float z[V], s[V], t[V], one[V];
    v_fma(z, xm, f.scale, f.bias);
    v_sigmoid(s, z);
    v_set(one, 1.f);
    v_sub(t, one, s);
    v_fma(t, z, t, one);
    v_mul(s, s, t);
    v_mul(dz, dy, s);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) dz[i] = dy[i];
  }
}
// Per-channel rstd of a run.
template <int V, class S>
DIT_DEV void spread(float (&d)[V], int c, int cpg, S value) {
  int g = c / cpg, left = cpg - (c - g * cpg);
  float t = value(g);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (left == 0) t = value(++g), left = cpg;
    --left;
    d[i] = t;
  }
}
// Sums of a thread.
template <int V>
struct GradSums {
  float A[V], B[V];
  DIT_DEV GradSums() { v_set(A, 0.f), v_set(B, 0.f); }
  DIT_DEV void add(const float (&dz)[V], const float (&xm)[V]) {
    v_add(A, A, dz);
    v_fma(B, dz, xm, B);
  }
};

// part[b, split, c] = (sum dz, sum dz xhat) over the split's pixels.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 3) gn_grad_sums_kernel(const __grid_constant__ GnParams P) {
  extern __shared__ float2 sm[];  // [rows][slab * V]
  start_next();
  const int64_t b = blockIdx.x / P.splits;
  const int split = blockIdx.x - b * P.splits;
  const int64_t p0 = range_begin(P.pixels, P.splits, split), p1 = range_begin(P.pixels, P.splits, split + 1);
  const Place at(P, V, blockIdx.y, p0, p1);
  const int width = P.slab * V;
  Affine<V> f;
  GradSums<V> S;
  if (at.on) {
    f.weights(P, at.c);
    f.statistics(at.c, P.cpg, [&](int g) { return make_float2(P.mean[b * P.groups + g], P.rstd[b * P.groups + g]); });
    walk2<T, V, kGradUnroll>(static_cast<const T*>(P.x) + b * P.xs[0] + at.p * P.xs[1] + at.c, at.rows * P.xs[1],
                             static_cast<const T*>(P.dy) + b * P.ds[0] + at.p * P.ds[1] + at.c, at.rows * P.ds[1],
                             at.count, [&](int, const Raw<T, V>& rx, const Raw<T, V>& rg) {
                               float v[V], g[V], xm[V], dz[V];
                               unpack<T, V>(rx, v);
                               unpack<T, V>(rg, g);
                               dz_of(f, v, g, P.act, xm, dz);
                               S.add(dz, xm);
                             });
    float r[V];
    spread(r, at.c, P.cpg, [&](int g) { return P.rstd[b * P.groups + g]; });
    v_mul(S.B, S.B, r);
  }
  add_rows<V>(at, S.A, S.B, sm, P.slab);
  const int c0 = blockIdx.y * width, here = min(width, P.channels - c0);
  float2* part = P.part + (b * P.splits + split) * P.channels + c0;
  for (int c = threadIdx.x; c < here; c += kThreads) part[c] = sm[pair_at(V, P.slab, c)];
}

DIT_DEV float block_sum(float v, float* sm) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) t += sm[i];
  return t;
}

// One (batch element, group): per-channel sums over the splits, and the
// group's s1, s2.  Threads (row, column): columns of channels, rows of splits.
__global__ void __launch_bounds__(kThreads) gn_grad_join_kernel(const __grid_constant__ GnParams P, int cols) {
  __shared__ float2 sm[kThreads];
  __shared__ float sums[kThreads / 32];
  start_next();
  const int64_t b = blockIdx.x / P.groups;
  const int g = blockIdx.x - b * P.groups;
  const int rows = kThreads / cols, col = threadIdx.x % cols, row = threadIdx.x / cols;
  const float2* part = P.part + b * P.splits * P.channels + (int64_t)g * P.cpg;
  float s1 = 0.f, s2 = 0.f;
  wait_previous();
  for (int c0 = 0; c0 < P.cpg; c0 += cols) {
    float A = 0.f, B = 0.f;
    if (c0 + col < P.cpg) {
#pragma unroll 4
      for (int s = row; s < P.splits; s += rows) {
        const float2 e = part[(int64_t)s * P.channels + c0 + col];
        A += e.x, B += e.y;
      }
    }
    sm[threadIdx.x] = make_float2(A, B);
    for (int h = rows / 2; h; h /= 2) {  // rows is a power of two
      __syncthreads();
      if (row < h) {
        const float2 o = sm[threadIdx.x + h * cols];
        A += o.x, B += o.y;
        sm[threadIdx.x] = make_float2(A, B);
      }
    }
    if (row == 0 && c0 + col < P.cpg) {
      const int c = g * P.cpg + c0 + col;
      P.chan[b * P.channels + c] = make_float2(A, B);
      const float w = P.w ? P.w[c] : 1.f;
      s1 = fmaf(w, A, s1), s2 = fmaf(w, B, s2);
    }
    __syncthreads();
  }
  const float total = (float)P.pixels * (float)P.cpg;
  s1 = block_sum(s1, sums);
  s2 = block_sum(s2, sums);
  if (threadIdx.x == 0) P.gsum[blockIdx.x] = P.pixels ? make_float2(s1 / total, s2 / total) : make_float2(0.f, 0.f);
}

// dw[c], db[c]: the channel sums over the batch, in order.
DIT_DEV void grad_weights(const GnParams& P, int c) {
  if (c >= P.channels) return;
  float A = 0.f, B = 0.f;
#pragma unroll 4
  for (int64_t b = 0; b < P.batch; ++b) {
    const float2 e = P.chan[b * P.channels + c];
    A += e.x, B += e.y;
  }
  if (P.db) P.db[c] = A;
  if (P.dw) P.dw[c] = B;
}
__global__ void __launch_bounds__(kThreads) gn_grad_weights_kernel(const __grid_constant__ GnParams P) {
  wait_previous();
  grad_weights(P, blockIdx.x * kThreads + threadIdx.x);
}

// dx = scale dz - c1 - xm c2 with c1 = rstd s1, c2 = rstd^2 s2.
template <int V>
struct GradApply {
  float c1[V], c2[V];
  template <class S>
  DIT_DEV void set(int c, int cpg, S value) {  // value(g) = (rstd, s1, s2)
    int g = c / cpg, left = cpg - (c - g * cpg);
    float3 t = value(g);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (left == 0) t = value(++g), left = cpg;
      --left;
      c1[i] = -t.x * t.y;
      c2[i] = -t.x * t.x * t.z;
    }
  }
  DIT_DEV void dx(const Affine<V>& f, const float (&xm)[V], float (&dz)[V]) const {
    float t[V];
    v_fma(t, xm, c2, c1);
    v_fma(dz, dz, f.scale, t);
  }
};

// dx; the blocks behind the last pixel range sum the channels over the batch.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 3) gn_grad_apply_kernel(const __grid_constant__ GnParams P) {
  const int64_t work = P.batch * P.passes;
  if (blockIdx.x >= work) {
    wait_previous();
    if (blockIdx.y == 0) grad_weights(P, (int)(blockIdx.x - work) * kThreads + threadIdx.x);
    return;
  }
  const int64_t at_block = work - 1 - blockIdx.x;
  const int64_t b = at_block / P.passes;
  const int split = at_block - b * P.passes;
  const int64_t p0 = range_begin(P.pixels, P.passes, split), p1 = range_begin(P.pixels, P.passes, split + 1);
  const Place at(P, V, blockIdx.y, p0, p1);
  Affine<V> f;
  GradApply<V> h;
  if (at.on) {
    f.weights(P, at.c);
    f.statistics(at.c, P.cpg, [&](int g) { return make_float2(P.mean[b * P.groups + g], P.rstd[b * P.groups + g]); });
  }
  wait_previous();
  if (!at.on) return;
  h.set(at.c, P.cpg, [&](int g) {
    const float2 s = P.gsum[b * P.groups + g];
    return make_float3(P.rstd[b * P.groups + g], s.x, s.y);
  });
  T* out = static_cast<T*>(P.out) + b * P.os[0] + at.p * P.os[1] + at.c;
  const int64_t ostep = at.rows * P.os[1];
  walk2<T, V, kGradUnroll>(static_cast<const T*>(P.x) + b * P.xs[0] + at.p * P.xs[1] + at.c, at.rows * P.xs[1],
                           static_cast<const T*>(P.dy) + b * P.ds[0] + at.p * P.ds[1] + at.c, at.rows * P.ds[1],
                           at.count, [&](int, const Raw<T, V>& rx, const Raw<T, V>& rg) {
                             float v[V], g[V], xm[V], dz[V];
                             unpack<T, V>(rx, v);
                             unpack<T, V>(rg, g);
                             dz_of(f, v, g, P.act, xm, dz);
                             h.dx(f, xm, dz);
                             store_f32<T, V>(out, dz);
                             out += ostep;
                           });
}

// One launch, as gn_cluster_kernel: x and dy stay in shared memory between
// the sums and dx.  With one batch element the channel sums are dw and db.
// Shared memory: sums [rows][slab * V] float2 (row 0 read by the cluster),
// chan[slab * V] float2, group sums [groups of the slab] float2, x, dy.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 2) gn_grad_cluster_kernel(const __grid_constant__ GnParams P, int data_elems) {
  extern __shared__ float4 raw_sm[];
  start_next();
  const int width = P.slab * V, rows = kThreads / P.slab, slab_groups = width / P.cpg;
  float2* sm = reinterpret_cast<float2*>(raw_sm);
  float2* chan = sm + rows * width;
  float2* gs = chan + width;
  T* data = reinterpret_cast<T*>(raw_sm) +
            ((reinterpret_cast<char*>(gs + slab_groups) - reinterpret_cast<char*>(raw_sm) + 15) / 16 * 16) / sizeof(T);

  const int rank = blockIdx.x % P.splits;
  const int64_t b = blockIdx.x / P.splits;
  const int64_t p0 = range_begin(P.pixels, P.splits, rank), p1 = range_begin(P.pixels, P.splits, rank + 1);
  const Place at(P, V, blockIdx.y, p0, p1);
  T* xm_ = data + threadIdx.x * V;
  T* gm_ = xm_ + data_elems;
  Affine<V> f;
  GradSums<V> S;
  if (at.on) {
    f.weights(P, at.c);
    f.statistics(at.c, P.cpg, [&](int g) { return make_float2(P.mean[b * P.groups + g], P.rstd[b * P.groups + g]); });
    walk2<T, V, kGradUnroll>(static_cast<const T*>(P.x) + b * P.xs[0] + at.p * P.xs[1] + at.c, at.rows * P.xs[1],
                             static_cast<const T*>(P.dy) + b * P.ds[0] + at.p * P.ds[1] + at.c, at.rows * P.ds[1],
                             at.count, [&](int i, const Raw<T, V>& rx, const Raw<T, V>& rg) {
                               float v[V], g[V], xm[V], dz[V];
                               store_raw<T, V>(xm_ + i * (kThreads * V), rx);
                               store_raw<T, V>(gm_ + i * (kThreads * V), rg);
                               unpack<T, V>(rx, v);
                               unpack<T, V>(rg, g);
                               dz_of(f, v, g, P.act, xm, dz);
                               S.add(dz, xm);
                             });
    float r[V];
    spread(r, at.c, P.cpg, [&](int g) { return P.rstd[b * P.groups + g]; });
    v_mul(S.B, S.B, r);
  }
  add_rows<V>(at, S.A, S.B, sm, P.slab);
  cluster_arrive();
  cluster_wait();
  const int c0 = blockIdx.y * width, here = min(width, P.channels - c0), groups = here / P.cpg, g0 = c0 / P.cpg;
  for (int c = threadIdx.x; c < here; c += kThreads) {
    float A = 0.f, B = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (r >= P.splits) continue;
      const float2 e = ld_cluster_f2(cluster_map(sm + pair_at(V, P.slab, c), r));
      A += e.x, B += e.y;
    }
    if (rank == 0) {
      if (P.chan) P.chan[b * P.channels + c0 + c] = make_float2(A, B);
      else {
        if (P.db) P.db[c0 + c] = A;
        if (P.dw) P.dw[c0 + c] = B;
      }
    }
    const float w = P.w ? P.w[c0 + c] : 1.f;
    chan[c] = make_float2(w * A, w * B);
  }
  __syncthreads();
  cluster_arrive();
  const float total = (float)P.pixels * (float)P.cpg;
  if (P.cpg <= 8) {
    for (int g = threadIdx.x; g < groups; g += kThreads) {
      float s1 = 0.f, s2 = 0.f;
      for (int c = 0; c < P.cpg; ++c) s1 += chan[g * P.cpg + c].x, s2 += chan[g * P.cpg + c].y;
      gs[g] = make_float2(s1 / total, s2 / total);
    }
  } else {
    const int lane = threadIdx.x & 31;
    for (int g = threadIdx.x >> 5; g < groups; g += kThreads / 32) {
      float s1 = 0.f, s2 = 0.f;
      for (int c = lane; c < P.cpg; c += 32) s1 += chan[g * P.cpg + c].x, s2 += chan[g * P.cpg + c].y;
      s1 = warp_sum(s1), s2 = warp_sum(s2);
      if (lane == 0) gs[g] = make_float2(s1 / total, s2 / total);
    }
  }
  __syncthreads();
  if (at.on) {
    GradApply<V> h;
    h.set(at.c, P.cpg, [&](int g) { return make_float3(P.rstd[b * P.groups + g], gs[g - g0].x, gs[g - g0].y); });
    T* out = static_cast<T*>(P.out) + b * P.os[0] + at.p * P.os[1] + at.c;
    const int64_t ostep = at.rows * P.os[1];
#pragma unroll 2
    for (int i = 0; i < at.count; ++i) {
      float v[V], g[V], xm[V], dz[V];
      unpack<T, V>(load_raw<T, V>(xm_ + i * (kThreads * V)), v);
      unpack<T, V>(load_raw<T, V>(gm_ + i * (kThreads * V)), g);
      dz_of(f, v, g, P.act, xm, dz);
      h.dx(f, xm, dz);
      store_f32<T, V>(out, dz);
      out += ostep;
    }
  }
  cluster_wait();
}

// ---------------------------------------------------------------- plan
int elem_bytes(int dtype) { return dtype == DIT_DTYPE_F32 ? 4 : 2; }

bool aligned(const void* p, const int64_t st[2], int elem, int to) {
  return !p || (((uintptr_t)p | (uintptr_t)(st[0] * elem) | (uintptr_t)(st[1] * elem)) & (to - 1)) == 0;
}

// Channels a thread takes: 16 bytes of them, or 4, or one.
int vec_of(const dit_group_norm_args& a) {
  const int e = elem_bytes(a.dtype);
  for (int to : {16, 4})
    if (a.channels % (to / e) == 0 && aligned(a.x, a.x_stride, e, to) && aligned(a.dy, a.dy_stride, e, to) &&
        aligned(a.out, a.out_stride, e, to))
      return to / e;
  return 1;
}

struct Plan {
  bool cluster;
  int vec, slab, nslab, splits, passes, unit;
  int data_elems;  // cluster form: elements of one staged tensor
  size_t smem;
};

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr int64_t kSmemMost = 200 << 10;

size_t scratch_bytes(const Plan& p, int cpg, bool backward) {
  const int rows = kThreads / p.slab, width = p.slab * p.vec;
  size_t n = (size_t)rows * width * 8;
  if (p.cluster) {
    n += backward ? (size_t)width * 8 + (size_t)(width / cpg) * 8 : kThreads * 4 + (size_t)(width / cpg) * 16;
    return (n + 15) / 16 * 16;
  }
  return n + (backward ? 0 : kThreads * 4);
}

// The three-launch form.
Plan split_plan(const dit_group_norm_args& a, int vec, bool backward) {
  Plan p{};
  p.vec = vec;
  const int cpg = a.channels / a.groups, runs = a.channels / vec, whole = cpg / gcd(cpg, vec);  // runs of whole groups
  p.slab = runs < kThreads ? runs : kThreads;
  if (runs > kThreads && whole <= kThreads) p.slab = kThreads / whole * whole;
  p.nslab = (int)ceil_div(runs, p.slab);
  // equal slabs of whole groups
  if (whole <= kThreads) {
    p.slab = (int)(ceil_div(ceil_div(runs, p.nslab), whole) * whole);
    p.nslab = (int)ceil_div(runs, p.slab);
  }
  p.unit = !backward && whole <= kThreads ? cpg : 1;
  const int rows = kThreads / p.slab;
  // pixel ranges: one wave of three blocks an SM, fewer where a thread would
  // have less than one batch of loads, more where it would sum over too many
  // pixels in a row for fp32 (the forward's sums are folded, the gradient's not)
  const int64_t each = a.batch * p.nslab;
  int64_t splits = 456 / each, most = a.pixels / ((int64_t)rows * kPassUnroll),
          least = ceil_div(a.pixels, (int64_t)rows * (backward ? 128 : 1024));
  if (splits > most) splits = most;
  if (splits < least) splits = least;
  p.splits = (int)(splits < 1 ? 1 : splits);
  int64_t passes = (backward ? 912 : 1216) / each;
  if (passes > most) passes = most;
  p.passes = (int)(passes < 1 ? 1 : passes);
  p.smem = scratch_bytes(p, cpg, backward);
  return p;
}

// The cluster form for a slab and cluster size; smem 0 where it does not fit.
Plan cluster_plan(const dit_group_norm_args& a, int vec, int slab, int blocks, bool backward) {
  Plan p{};
  p.cluster = true;
  p.vec = vec;
  p.slab = slab;
  p.nslab = (int)ceil_div(a.channels / vec, slab);
  p.splits = blocks;
  p.unit = a.channels / a.groups;
  const int rows = kThreads / slab;
  const int64_t iters = ceil_div(ceil_div(a.pixels, blocks), rows);
  const int64_t data = iters * kThreads * vec * elem_bytes(a.dtype);
  if (data > kSmemMost) return p;
  const size_t smem = scratch_bytes(p, p.unit, backward) + (size_t)data * (backward ? 2 : 1);
  if (smem > (size_t)kSmemMost) return p;
  p.data_elems = (int)(iters * kThreads * vec);
  p.smem = smem;
  return p;
}

Plan plan_of(const dit_group_norm_args& a, int vec, bool backward) {
  if (getenv("GN_CLUSTER")) {  // EXPERIMENT
    int slab, blocks;
    sscanf(getenv("GN_CLUSTER"), "%d,%d", &slab, &blocks);
    const int cpg = a.channels / a.groups, whole = cpg / gcd(cpg, vec);
    slab = (slab + whole - 1) / whole * whole;
    if (slab > a.channels / vec) slab = a.channels / vec;
    if (slab <= kThreads && a.pixels) {
      Plan p = cluster_plan(a, vec, slab, blocks, backward);
      if (p.smem) return p;
    }
  }
  return split_plan(a, vec, backward);
}

int64_t round256(int64_t n) { return (n + 255) & ~(int64_t)255; }

// Workspace of a plan: partials, then [batch, groups] pairs, then channel sums.
int64_t part_bytes(const dit_group_norm_args& a, const Plan& p) {
  return p.cluster ? 0 : round256(a.batch * p.splits * (int64_t)(a.channels / p.unit) * 8);
}
int64_t group_bytes(const dit_group_norm_args& a, const Plan& p) { return p.cluster ? 0 : round256(a.batch * a.groups * 8); }
int64_t chan_bytes(const dit_group_norm_args& a, const Plan& p, bool backward) {
  return !backward || (p.cluster && a.batch == 1) ? 0 : round256(a.batch * (int64_t)a.channels * 8);
}

// ---------------------------------------------------------------- launch
#define GN_TRY(expr)                      \
  do {                                    \
    const cudaError_t e_ = (expr);        \
    if (e_ != cudaSuccess) return e_;     \
  } while (0)

template <typename T, int V>
cudaError_t run(const dit_group_norm_args& a, const Plan& pl, const GnParams& P, bool backward, cudaStream_t s) {
  const dim3 grid((unsigned)(a.batch * pl.splits), (unsigned)pl.nslab);
  const dim3 pass((unsigned)(a.batch * pl.passes), (unsigned)pl.nslab), bg((unsigned)(a.batch * a.groups));
  const unsigned extra = P.dw || P.db ? (unsigned)ceil_div(a.channels, kThreads) : 0;
  if (pl.cluster) {
    if (!backward) return launch_kernel(gn_cluster_kernel<T, V>, grid, kThreads, pl.smem, s, pl.splits, false, P);
    GN_TRY(launch_kernel(gn_grad_cluster_kernel<T, V>, grid, kThreads, pl.smem, s, pl.splits, false, P, pl.data_elems));
    return extra && a.batch > 1 ? launch_kernel(gn_grad_weights_kernel, dim3(extra), kThreads, 0, s, 1, true, P) : cudaSuccess;
  }
  if (!backward) {
    GN_TRY(launch_kernel(gn_sums_kernel<T, V>, grid, kThreads, pl.smem, s, 1, false, P));
    GN_TRY(launch_kernel(gn_join_kernel, bg, kJoinThreads, 0, s, 1, true, P));
    return a.pixels ? launch_kernel(gn_apply_kernel<T, V>, pass, kThreads, 0, s, 1, true, P) : cudaSuccess;
  }
  int cols = 1;
  while (cols < P.cpg && cols < 32) cols *= 2;
  GN_TRY(launch_kernel(gn_grad_sums_kernel<T, V>, grid, kThreads, pl.smem, s, 1, false, P));
  GN_TRY(launch_kernel(gn_grad_join_kernel, bg, kThreads, 0, s, 1, true, P, cols));
  return launch_kernel(gn_grad_apply_kernel<T, V>, dim3(pass.x + extra, pass.y), kThreads, 0, s, 1, true, P);
}

template <typename T>
cudaError_t run_vec(const dit_group_norm_args& a, const Plan& pl, const GnParams& P, bool backward, cudaStream_t s) {
  constexpr int most = 16 / sizeof(T);
  if (pl.vec == most) return run<T, most>(a, pl, P, backward, s);
  if constexpr (sizeof(T) == 2)
    if (pl.vec == 2) return run<T, 2>(a, pl, P, backward, s);
  return run<T, 1>(a, pl, P, backward, s);
}

}  // namespace

int64_t group_norm_workspace(const dit_group_norm_args& a, bool backward) {
  if (a.batch == 0) return 0;
  // enough for any alignment of the tensors
  int64_t need = 0;
  for (int vec : {16 / elem_bytes(a.dtype), 4 / elem_bytes(a.dtype), 1}) {
    if (a.channels % vec) continue;
    const Plan p = plan_of(a, vec, backward);
    const int64_t n = part_bytes(a, p) + group_bytes(a, p) + chan_bytes(a, p, backward);
    if (n > need) need = n;
  }
  return need;
}

cudaError_t group_norm_run(const dit_group_norm_args& a, bool backward, float* workspace, cudaStream_t stream) {
  if (a.batch == 0) {
    // nothing was summed
    for (float* d : {a.dweight, a.dbias})
      if (backward && d) GN_TRY(cudaMemsetAsync(d, 0, (size_t)a.channels * sizeof(float), stream));
    return cudaSuccess;
  }
  GnParams P{};
  const Plan pl = plan_of(a, vec_of(a), backward);
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
  P.passes = pl.passes;
  P.slab = pl.slab;
  P.unit = pl.unit;
  P.act = a.act;
  P.eps = a.eps;
  P.w = a.weight;
  P.b = a.bias;
  P.dw = a.dweight;
  P.db = a.dbias;
  char* ws = reinterpret_cast<char*>(workspace);
  P.part = reinterpret_cast<float2*>(ws);
  ws += part_bytes(a, pl);
  float* bg = reinterpret_cast<float*>(ws);
  ws += group_bytes(a, pl);
  if (!backward) {
    P.mean_out = a.mean;
    P.rstd_out = a.rstd;
    if (!pl.cluster) {
      if (!a.mean) P.mean_out = bg;
      if (!a.rstd) P.rstd_out = bg + a.batch * a.groups;
    }
    P.mean = P.mean_out;
    P.rstd = P.rstd_out;
  } else {
    P.mean = a.mean;
    P.rstd = a.rstd;
    P.gsum = reinterpret_cast<float2*>(bg);
    P.chan = chan_bytes(a, pl, backward) ? reinterpret_cast<float2*>(ws) : nullptr;
  }
  if (a.dtype == DIT_DTYPE_F32) return run_vec<float>(a, pl, P, backward, stream);
  if (a.dtype == DIT_DTYPE_BF16) return run_vec<__nv_bfloat16>(a, pl, P, backward, stream);
  return run_vec<__half>(a, pl, P, backward, stream);
}

}  // namespace dit
