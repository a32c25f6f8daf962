// Group norm of channels-last activations with an optional SiLU, and its
// gradient.
//
// Mathematics.  Per batch element and group: mean and population variance over
// pixels x channels, xhat = (x - mean) rstd, z = xhat w + b, y = act(z).
// Gradient: dz = dy act'(z); per channel A = sum dz, B = sum dz xhat over the
// pixels; dw = sum_batch B, db = sum_batch A; with the group means
// s1 = mean(w dz), s2 = mean(w dz xhat): dx = rstd (w dz - s1 - xhat s2).
//
// Sums.  A thread owns a run of V channels and walks pixels, summing x - K and
// (x - K)^2 per channel about the block's pivot K, the median of three of the
// channel's pixels in the block: the sums are of deviations, so nothing
// cancels however large the mean, and a single outlier cannot become the
// pivot.  Threads are joined by plain sums, then turned into (mean, M2) about
// the mean, and channels of a group and blocks joined as (count, mean, M2), all
// in a fixed order: results are the same bits every time.  The joined means are
// unevaluated sums of two floats until the last step, so a group's mean is as good
// where its channels' means cancel.
//
// What bounds it: HBM and the second look at x.  Two forms:
//   - whole groups of a batch element that fit a cluster's shared memory: one
//     launch.  A block loads its pixels once, into shared memory, the cluster
//     joins the groups' sums through distributed shared memory, and the block
//     writes its pixels out of shared memory: one read, one write.
//   - otherwise sums per (share of the pixels, group), a join per (batch
//     element, group) where the shares are many, and a pass that walks the
//     pixels backwards, so that what the sums read last is still in L2;
//     launches chained by programmatic dependence, the pass's first loads on
//     their way before the sums are done.
// Measured on one GB300 (bf16): 1024 x 1024 pixels x 128 channels with SiLU 132 us:
// the sums 55 us for 328 MB of DRAM traffic (60 of them the previous output on its
// way out), the pass 78 us for 395 MB, 80 MB of x out of L2 (reading L2 and writing
// DRAM 5 TB/s of writes, both from DRAM 3.1, so 76 us is what that traffic takes).
// 21 x 6240 x 384 50.0 us; gradient of 4 x 16384 x 512 53.0 us.  Blocks that each
// take one range of pixels instead of turns leave only 11 MB of x in L2 (137 us);
// register loads instead of rings 136 us; normal stores 134 us.
#include "launch.cuh"
#include "operators.h"
#include "vec.cuh"

namespace dit {

namespace {

constexpr int kThreads = 256;
// Blocks an SM of the kernels that stream a tensor: two or four, whose
// shared-memory rings keep about 110 KB on its way; five or six where runs are
// shorter than 8 bytes and loads go to registers.
constexpr int stream_blocks(int run_bytes) { return run_bytes == 16 ? 2 : run_bytes == 8 ? 4 : run_bytes == 4 ? 5 : 6; }

struct GnParams {
  const void* x;
  const void* dy;
  void* out;
  int64_t xs[2], ds[2], os[2];
  int64_t batch;
  int pixels, channels, groups, cpg;
  int splits;      // blocks that share a batch element's pixels
  int passes;      // the same for the pass that writes
  int whole_batch; // gradient on clusters that hold the whole batch
  int slab;        // runs of V channels a block covers
  int part_lanes;  // threads that sum one channel's rows: a power of two
  int unit;        // channels of one partial: cpg where slabs hold whole groups, else 1
  int fold;        // the forward's pass joins the partials itself
  int act;
  float eps;
  const float* w;
  const float* b;
  const float* mean;  // [batch, groups], read
  const float* rstd;
  float* mean_out;    // [batch, groups], written, or NULL (cluster form)
  float* rstd_out;
  float4* sums;       // forward [batch, splits, channels / unit]: Joint as (n, mean, low, M)
  float2* part;       // gradient [batch, splits, channels]
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
DIT_DEV void v_fms(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
  each<V>([&](int i) {
            const float2 r = ffma2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(-c[i], -c[i + 1]));
            d[i] = r.x, d[i + 1] = r.y;
          },
          [&](int i) { d[i] = fmaf(a[i], b[i], -c[i]); });
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
// sigma(z) and its derivative sigma (1 - sigma).  For fp32 activations from e =
// 2^(-|z| log2 e) in (0, 1] and r = 1 / (1 + e): e r or r, and e r^2.  What the
// exponent's rounding and log2 e's own leave out goes back in as a factor 1 + low
// ln 2, so each is within 16 x 2^-24 of itself however far z is from 0, until e
// is below 2^-126 and taken as 0 (ex2 4 x 2^-24, the reciprocal 2, six roundings).
// For 16-bit activations 1 / (1 + 2^(-z log2 e)) without that: the exponent's
// rounding gives |z| 2^-24 relative, the constant's a quarter of that, the rest
// 2^-21; at most 2^-17 where the result is rounded to 2^-9 or 2^-12 of itself.
// With the factor there the 1048576 x 128 map took 136.0 us instead of 129.7 and
// its gradient 241 instead of 215; in fp32 512 x 512 x 128 took 61.6 instead of
// 61.2, its gradient 108.8 instead of 104.2.
template <typename T, int V>
DIT_DEV void v_sigmoid(float (&d)[V], float (&c)[V], const float (&z)[V]) {
  if constexpr (sizeof(T) == 4) {
    float u[V], k[V], k_low[V], ln2[V], one[V], t[V], low[V];
    v_set(k, 1.4426950216293335f);       // log2 e in two parts
    v_set(k_low, 1.9259629911266175e-8f);
    v_set(ln2, 0.6931471805599453f);
    v_set(one, 1.f);
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = -fminf(fabsf(z[i]), 150.f);
    v_mul(t, u, k);
    v_fms(low, u, k, t);
    v_fma(low, u, k_low, low);
    v_fma(low, low, ln2, one);
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = ex2_approx(t[i]);
    v_mul(t, t, low);
    v_add(u, t, one);
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = rcp_approx(u[i]);
    v_mul(t, t, u);
    v_mul(c, t, u);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = z[i] < 0.f ? t[i] : u[i];
  } else {
    float k[V], one[V], t[V];
    v_set(k, -1.4426950408889634f);
    v_set(one, 1.f);
    v_mul(t, z, k);
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = ex2_approx(t[i]);
    v_add(t, t, one);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = rcp_approx(t[i]);
    v_sub(c, one, d);
    v_mul(c, c, d);
  }
}

// ---------------------------------------------------------------- blocks
// ceil(n / step): the sum passes 31 bits near 2^31 pixels
DIT_DEV int steps_from(int n, int step) { return (int)(((unsigned)n + (unsigned)step - 1) / (unsigned)step); }
// `shares` blocks take a batch element's pixels in turn, `rows` at a time: at
// any moment all of them are near the same place, so what was read last is the
// end of the tensor.
// Thread (row, run) of share s takes run `run` of the slab and pixels
// p, p + step, ...
struct Place {
  int rows, row, run, c, p, step, count;
  bool on;
  DIT_DEV Place(const GnParams& P, int V, int slab_index, int s, int shares) {
    rows = kThreads / (unsigned)P.slab;
    row = threadIdx.x / (unsigned)P.slab;
    run = threadIdx.x - row * P.slab;
    c = (slab_index * P.slab + run) * V;
    on = row < rows && c < P.channels;
    step = shares * rows;
    p = s * rows + row;
    count = on && p < P.pixels ? steps_from(P.pixels - p, step) : 0;
  }
};
// Pixels of share s.
DIT_DEV int share_pixels(const GnParams& P, int rows, int s, int shares) {
  const int turns = P.pixels / (unsigned)(shares * rows), left = P.pixels - turns * shares * rows - s * rows;
  return turns * rows + (left < 0 ? 0 : left < rows ? left : rows);
}

// B bytes (4, 8 or 16) to shared memory in the background.
template <int B>
DIT_DEV void async_copy(void* dst, const void* src) {
  if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(B) : "memory");
}
template <int B>
DIT_DEV void async_copy(void* dst, const void* src, uint64_t policy) {
  if constexpr (B == 16)
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "l"(policy) : "memory");
  else
    asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(B), "l"(policy) : "memory");
}

// A thread's pixels 0 .. count - 1 of N tensors, read ahead of their use: run(
// body) calls body(i, raw[N]) for each.  Runs of 16 or 8 bytes come through a ring
// in shared memory by cp.async, STAGES batches of U pixels, each thread filling
// and reading its own slots only (no barriers, no registers held by what is on
// its way); a slot is filled again one batch after its values were used.
// Shorter runs are loaded into registers a batch ahead: cp.async cannot move 2
// bytes, and with 4 it measured 6 % slower than registers.
// LAST: the data is not read again (first out of L2).
template <typename T, int V, int N, int U, int STAGES, bool LAST>
struct Feed {
  enum : int {
    kRun = V * (int)sizeof(T),
    kRing = kRun >= 8,
    kWhole = !kRing && (N == 1 || kRun == 2),  // instructions count there: whole batches go without checks
    kSlot = kRing ? kThreads * V : 0,  // elements of a slot of all threads
    kBytes = STAGES * U * N * kSlot * (int)sizeof(T)
  };
  const T* src[N];
  int64_t step[N];
  T* ring;
  int count, next, slot;
  uint64_t policy;
  Raw<T, V> reg[kRing ? 1 : U * N];

  DIT_DEV void from(int k, const T* p, int64_t s) { src[k] = p, step[k] = s; }
  DIT_DEV void fetch_one(int u) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const T* p = src[k] + u * step[k];
      if constexpr (kRing) copy(ring + ((slot * U + u) * N + k) * kSlot, p);
      else reg[u * N + k] = load_raw<T, V>(p);
    }
  }
  DIT_DEV void fetch() {  // the next batch
    if (kWhole && next + U <= count) {
#pragma unroll
      for (int u = 0; u < U; ++u) fetch_one(u);
    } else {
#pragma unroll
      for (int u = 0; u < (kWhole ? U - 1 : U); ++u)
        if (next + u < count) fetch_one(u);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) src[k] += U * step[k];
    next += U;
    if constexpr (kRing) {
      asm volatile("cp.async.commit_group;" ::: "memory");
      slot = slot + 1 == STAGES ? 0 : slot + 1;
    }
  }
  DIT_DEV void copy(T* dst, const T* p) const {
    if constexpr (LAST) async_copy<kRun>(dst, p, policy);
    else async_copy<kRun>(dst, p);
  }
  // the first loads on their way; `ring_` is the block's, kBytes of it
  DIT_DEV void start(void* ring_, int count_) {
    ring = static_cast<T*>(ring_) + threadIdx.x * V;
    count = count_;
    next = slot = 0;
    if constexpr (LAST) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    if constexpr (kRing) {
#pragma unroll
      for (int k = 0; k < STAGES - 1; ++k) fetch();
    } else {
      fetch();
    }
  }
  template <class Body>
  DIT_DEV void run(Body body) {
    int at = 0;
    for (int i = 0; i < count; i += U) {
      Raw<T, V> r[U][N];
      if constexpr (kRing) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int k = 0; k < N; ++k) r[u][k] = load_raw<T, V>(ring + ((at * U + u) * N + k) * kSlot);
        at = at + 1 == STAGES ? 0 : at + 1;
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int k = 0; k < N; ++k) r[u][k] = reg[u * N + k];
      }
      fetch();
      if (kWhole && i + U <= count) {
#pragma unroll
        for (int u = 0; u < U; ++u) body(i + u, r[u]);
      } else {
#pragma unroll
        for (int u = 0; u < (kWhole ? U - 1 : U); ++u)
          if (i + u < count) body(i + u, r[u]);
      }
    }
  }
};
template <typename T, int V, bool LAST>
using Feed1 = Feed<T, V, 1, (V * sizeof(T) >= 8 ? 2 : 8), 8, LAST>;
template <typename T, int V, bool LAST>
using Feed2 = Feed<T, V, 2, (V * sizeof(T) >= 8 ? 1 : V * sizeof(T) == 4 ? 4 : 8), 8, LAST>;

// A thread's sums of x - K and (x - K)^2 per channel.
template <int V>
struct Moments {
  float K[V], s[V], q[V];
  DIT_DEV Moments() { v_set(K, 0.f), v_set(s, 0.f), v_set(q, 0.f); }
  // median of three of the block's pixels: row 0's first, middle and last
  template <typename T>
  DIT_DEV void pivot(const T* first, int64_t step, int count) {
    const Raw<T, V> r[3] = {load_raw<T, V>(first), load_raw<T, V>(first + count / 2 * step),
                            load_raw<T, V>(first + (count - 1) * step)};
    float a[V], b[V], c[V];
    unpack<T, V>(r[0], a);
    unpack<T, V>(r[1], b);
    unpack<T, V>(r[2], c);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float m = fmaxf(fminf(a[i], b[i]), fminf(fmaxf(a[i], b[i]), c[i]));
      K[i] = fabsf(m) <= 3.402823466e38f ? m : 0.f;
    }
  }
  DIT_DEV void add(const float (&v)[V]) {
    float d[V];
    v_sub(d, v, K);
    v_add(s, s, d);
    v_fma(q, d, d, q);
  }
};

// Per-channel pairs of a block's rows in shared memory, [rows][V][slab] and a
// pair of padding a row: neither the writers (runs next to each other) nor the
// readers (rows or channels next to each other) meet on a bank.
// Sums the rows' pairs: out(c, total) once for every channel c of the slab, by
// `part` neighbouring threads a channel.
template <int V, class Out>
DIT_DEV void sum_rows(const Place& at, const float (&A)[V], const float (&B)[V], float2* sm, int slab, int part, Out out) {
  const int width = slab * V, pitch = width + 1;
  if (at.row < at.rows) {
#pragma unroll
    for (int i = 0; i < V; ++i) sm[at.row * pitch + i * slab + at.run] = make_float2(A[i], B[i]);
  }
  __syncthreads();
  const int t = threadIdx.x & (part - 1), per = kThreads / (unsigned)part;
  for (int c0 = 0; c0 < width; c0 += per) {
    const int j = c0 + threadIdx.x / (unsigned)part;  // place in a row: channel run j % slab, element j / slab
    float2 v = make_float2(0.f, 0.f);
    if (j < width)
      for (int r = t; r < at.rows; r += part) {
        const float2 o = sm[r * pitch + j];
        v.x += o.x, v.y += o.y;
      }
    for (int o = part >> 1; o; o >>= 1) {
      v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
      v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
    }
    if (t == 0 && j < width) out(j % (unsigned)slab * V + j / (unsigned)slab, v);
  }
  __syncthreads();
}

DIT_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// A mean as the unevaluated sum of two floats, and the second moment about it.
struct Mom {
  float mean, low, M;
};
// mean + low of a sum of n values given as h + l.
DIT_DEV float2 mean_of(float h, float l, float n) {
  const float m = h / n;
  return make_float2(m, isfinite(m) ? (fmaf(-m, n, h) + l) / n : 0.f);
}

// Joins the channels of every group of the slab, each of `len` pixels, from
// their moments in ch; out(g, Mom).  A thread a group of few channels, a warp
// one of many.
template <class Out>
DIT_DEV void join_channels(const Mom* ch, int groups, int cpg, float len, Out out) {
  const int lanes = cpg <= 8 ? 1 : 32, lane = cpg <= 8 ? 0 : threadIdx.x & 31;
  for (int g = threadIdx.x / (unsigned)lanes; g < groups; g += kThreads / lanes) {
    const Mom* e = ch + g * cpg;
    float h = 0.f, l = 0.f, M = 0.f, t;
    for (int c = lane; c < cpg; c += lanes) {
      h = two_sum(h, e[c].mean, t);
      l += t + e[c].low;
    }
    if (lanes > 1) {
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float oh = __shfl_xor_sync(0xFFFFFFFFu, h, o), ol = __shfl_xor_sync(0xFFFFFFFFu, l, o);
        h = two_sum(h, oh, t);
        l += ol + t;
      }
    }
    const float2 m = mean_of(h, l, (float)cpg);
    for (int c = lane; c < cpg; c += lanes) {
      const float d = (e[c].mean - m.x) + (e[c].low - m.y);
      M += fmaf(len * d, d, e[c].M);
    }
    if (lanes > 1) M = warp_sum(M);
    if (lane == 0) out(g, Mom{m.x, m.y, M});
  }
}

// Moments of two sets joined into the first.
struct Joint {
  float n, mean, low, M;
  DIT_DEV void take(float on, float omean, float olow, float oM) {
    if (on == 0.f) return;
    if (n == 0.f) {
      n = on, mean = omean, low = olow, M = oM;
      return;
    }
    const float f = on / (n + on), d = (omean - mean) + (olow - low);
    float t;
    if (!isfinite(d)) {  // a mean that is infinite stays so; no variance about it
      n += on, mean += omean, low = 0.f, M = d - d;
      return;
    }
    M += fmaf(d * d, n * f, oM);
    mean = two_sum(mean, d * f, t);
    low += t;
    n += on;
  }
  DIT_DEV void take(const float4& o) { take(o.x, o.y, o.z, o.w); }
  // of the lane `o` further on, where there is one
  DIT_DEV void take_down(int o, bool some) {
    const float4 v = make_float4(__shfl_down_sync(0xFFFFFFFFu, n, o), __shfl_down_sync(0xFFFFFFFFu, mean, o),
                                 __shfl_down_sync(0xFFFFFFFFu, low, o), __shfl_down_sync(0xFFFFFFFFu, M, o));
    if (some) take(v);
  }
  DIT_DEV float4 packed() const { return make_float4(n, mean, low, M); }
  DIT_DEV float rounded_mean() const { return isfinite(mean) ? mean + low : mean; }
};

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
template <typename T, int V>
DIT_DEV void activate(float (&v)[V], int act) {
  if (act == DIT_ACT_SILU) {
    float s[V], c[V];
    v_sigmoid<T>(s, c, v);
    v_mul(v, v, s);
  }
}

// ---------------------------------------------------------------- forward, two or three launches
// Every channel's moments over the block's `len` pixels, into ch.  drain(A)
// runs the thread's pixels through A; ch and piv are [slab * V].
template <typename T, int V, class Drain>
DIT_DEV void block_moments(const GnParams& P, const Place& at, const T* x, int len, float2* sm, Mom* ch, float* piv,
                           Drain drain) {
  Moments<V> A;
  if (at.on && len > 0) {
    const T* row0 = x + (at.p - at.row) * P.xs[1] + at.c;
    A.pivot(row0, at.step * P.xs[1], steps_from(P.pixels - (at.p - at.row), at.step));
    if (at.row == 0)
#pragma unroll
      for (int i = 0; i < V; ++i) piv[at.run * V + i] = A.K[i];
    drain(A);
  }
  const float n = (float)len, in = len > 0 ? 1.f / n : 0.f;
  sum_rows<V>(at, A.s, A.q, sm, P.slab, P.part_lanes, [&](int c, float2 v) {
    const float d = v.x * in;
    Mom m{0.f, 0.f, fmaf(-d, v.x, v.y)};
    if (len > 0) m.mean = two_sum(piv[c], d, m.low);
    ch[c] = m;
  });
}

// sums[b, split, unit] = moments of the unit's channels over the split.
// Shared memory: the ring, sums [rows][slab * V + 1] float2, ch [slab * V] Mom,
// piv [slab * V].
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, stream_blocks(V * sizeof(T))) gn_sums_kernel(const __grid_constant__ GnParams P) {
  extern __shared__ float4 raw_sm[];
  using F = Feed1<T, V, false>;
  float2* sm = reinterpret_cast<float2*>(reinterpret_cast<char*>(raw_sm) + F::kBytes);
  start_next();
  const uint32_t b = blockIdx.x / (uint32_t)P.splits, split = blockIdx.x - b * P.splits;
  const Place at(P, V, blockIdx.y, split, P.splits);
  const T* x = static_cast<const T*>(P.x) + b * P.xs[0];
  F feed;
  feed.from(0, x + at.p * P.xs[1] + at.c, at.step * P.xs[1]);
  feed.start(raw_sm, at.count);
  const int len = share_pixels(P, at.rows, split, P.splits);
  const int width = P.slab * V, c0 = blockIdx.y * width;
  Mom* ch = reinterpret_cast<Mom*>(sm + at.rows * (width + 1));
  block_moments<T, V>(P, at, x, len, sm, ch, reinterpret_cast<float*>(ch + width), [&](Moments<V>& A) {
    feed.run([&](int, const Raw<T, V>(&r)[1]) {
      float v[V];
      unpack<T, V>(r[0], v);
      A.add(v);
    });
  });
  const int here = min(width, P.channels - c0);
  float4* sums = P.sums + ((int64_t)blockIdx.x * P.channels + c0) / P.unit;
  const float n = (float)len * (float)P.unit;
  if (P.unit == 1) {
    for (int c = threadIdx.x; c < here; c += kThreads) sums[c] = make_float4(n, ch[c].mean, ch[c].low, ch[c].M);
  } else {
    join_channels(ch, here / P.cpg, P.cpg, (float)len, [&](int g, Mom m) { sums[g] = make_float4(n, m.mean, m.low, m.M); });
  }
}

// Joins the partials of one (batch element, group).
constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads) gn_join_kernel(const __grid_constant__ GnParams P) {
  __shared__ Joint sm[kJoinThreads / 32];
  start_next();
  const uint32_t b = blockIdx.x / (uint32_t)P.groups;
  const int g = blockIdx.x - b * P.groups;
  const int per = P.cpg / P.unit, stride = P.channels / P.unit;
  const float4* sums = P.sums + (int64_t)b * P.splits * stride + (int64_t)g * per;
  const int64_t entries = (int64_t)P.splits * per;
  Joint J{0.f, 0.f, 0.f, 0.f};
  wait_previous();
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < entries; i += kJoinThreads) {
    const int s = per == 1 ? (int)i : (int)(i / per);
    J.take(sums[(int64_t)s * stride + (i - (int64_t)s * per)]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) J.take_down(o, true);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = J;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < kJoinThreads / 32; ++i) J.take(sm[i].packed());
    P.mean_out[blockIdx.x] = J.rounded_mean();
    P.rstd_out[blockIdx.x] = rstd_of(J.n > 0.f ? J.M / J.n : 0.f, P.eps);
  }
}

// `lanes` (a power of two) neighbouring threads join one group's partials of a
// batch element: stat[g] = (mean, rstd) of the slab's groups.
DIT_DEV void fold_groups(const GnParams& P, uint32_t b, int g0, int groups, float2* stat, bool write) {
  int lanes = 1;
  while (lanes < 32 && 2 * lanes * groups <= kThreads) lanes *= 2;
  const int t = threadIdx.x & (lanes - 1), per = kThreads / (unsigned)lanes;
  const float4* sums = P.sums + (int64_t)b * P.splits * P.groups + g0;
  for (int base = 0; base < groups; base += per) {
    const int g = base + threadIdx.x / (unsigned)lanes;
    Joint J{0.f, 0.f, 0.f, 0.f};
    if (g < groups) {
#pragma unroll 4
      for (int s = t; s < P.splits; s += lanes) J.take(sums[(int64_t)s * P.groups + g]);
    }
    for (int o = lanes >> 1; o; o >>= 1) J.take_down(o, t + o < lanes);
    if (t == 0 && g < groups) {
      const float mean = J.rounded_mean(), rstd = rstd_of(J.n > 0.f ? J.M / J.n : 0.f, P.eps);
      stat[g] = make_float2(mean, rstd);
      if (write) {
        const int64_t bg = (int64_t)b * P.groups + g0 + g;
        if (P.mean_out) P.mean_out[bg] = mean;
        if (P.rstd_out) P.rstd_out[bg] = rstd;
      }
    }
  }
  __syncthreads();
}

// Shared memory: the ring, then stat [groups of the slab] float2 (P.fold).
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, stream_blocks(V * sizeof(T))) gn_apply_kernel(const __grid_constant__ GnParams P) {
  extern __shared__ float4 raw_sm[];
  using F = Feed1<T, V, true>;
  float2* stat = reinterpret_cast<float2*>(reinterpret_cast<char*>(raw_sm) + F::kBytes);
  const uint32_t b = blockIdx.x / (uint32_t)P.passes, share = blockIdx.x - b * P.passes;
  const Place at(P, V, blockIdx.y, share, P.passes);
  // backwards: what the sums read last first.  x is nobody's output, so its
  // loads need not wait for the sums.
  const int64_t last = at.p + (int64_t)(at.count - 1) * at.step, ystep = -at.step * P.os[1];
  F feed;
  feed.from(0, static_cast<const T*>(P.x) + b * P.xs[0] + last * P.xs[1] + at.c, -at.step * P.xs[1]);
  feed.start(raw_sm, at.count);
  Affine<V> f;
  if (at.on) f.weights(P, at.c);
  wait_previous();
  if (P.fold) {
    const int width = P.slab * V, c0 = blockIdx.y * width, g0 = c0 / P.cpg, groups = min(width, P.channels - c0) / P.cpg;
    fold_groups(P, b, g0, groups, stat, share == 0);
    if (at.on) f.statistics(at.c, P.cpg, [&](int g) { return stat[g - g0]; });
  } else if (at.on) {
    f.statistics(at.c, P.cpg, [&](int g) { return make_float2(P.mean[(int64_t)b * P.groups + g], P.rstd[(int64_t)b * P.groups + g]); });
  }
  T* y = static_cast<T*>(P.out) + b * P.os[0] + last * P.os[1] + at.c;
  feed.run([&](int, const Raw<T, V>(&r)[1]) {
    float v[V];
    unpack<T, V>(r[0], v);
    f.z(v);
    activate<T>(v, P.act);
    store_f32_stream<T, V>(y, v);
    y += ystep;
  });
}

// ---------------------------------------------------------------- forward, one launch
// All of a thread's pixels into its own places of shared memory, [i][thread]:
// in the background where cp.async can (staged() waits), else batch by batch.
template <typename T, int V>
DIT_DEV void stage(T* mine, const T* x, int64_t step, int count) {
  if constexpr (V * sizeof(T) >= 4) {
    for (int i = 0; i < count; ++i, x += step) async_copy<V * sizeof(T)>(mine + i * (kThreads * V), x);
  } else {
#pragma unroll 4
    for (int i = 0; i < count; ++i, x += step) mine[i * (kThreads * V)] = *x;
  }
}
DIT_DEV void staged() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A cluster of `splits` blocks takes one slab (whole groups) of one batch
// element; each block keeps its pixels in shared memory, every thread reading
// back only what it wrote itself.
// Shared memory: own [groups of the slab] float4 (read by the cluster), stat
// [groups of the slab] float2, sums, ch and piv as gn_sums_kernel, data.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 2) gn_cluster_kernel(const __grid_constant__ GnParams P) {
  extern __shared__ float4 raw_sm[];
  const int width = P.slab * V, rows = kThreads / (unsigned)P.slab, slab_groups = width / P.cpg;
  float4* own = raw_sm;
  float2* stat = reinterpret_cast<float2*>(own + slab_groups);
  float2* sm = stat + slab_groups;
  Mom* ch = reinterpret_cast<Mom*>(sm + rows * (width + 1));
  float* piv = reinterpret_cast<float*>(ch + width);
  T* data = reinterpret_cast<T*>(raw_sm) +
            ((reinterpret_cast<char*>(piv + width) - reinterpret_cast<char*>(raw_sm) + 15) / 16 * 16) / sizeof(T);

  const uint32_t b = blockIdx.x / (uint32_t)P.splits;
  const int rank = blockIdx.x - b * P.splits;
  const Place at(P, V, blockIdx.y, rank, P.splits);
  const int len = share_pixels(P, rows, rank, P.splits);
  T* mine = data + threadIdx.x * V;
  Affine<V> f;
  if (at.on) f.weights(P, at.c);
  const T* x = static_cast<const T*>(P.x) + b * P.xs[0];
  stage<T, V>(mine, x + at.p * P.xs[1] + at.c, at.step * P.xs[1], at.count);
  block_moments<T, V>(P, at, x, len, sm, ch, piv, [&](Moments<V>& A) {
    staged();
#pragma unroll 4
    for (int i = 0; i < at.count; ++i) {
      float v[V];
      unpack<T, V>(load_raw<T, V>(mine + i * (kThreads * V)), v);
      A.add(v);
    }
  });
  const int c0 = blockIdx.y * width, groups = min(width, P.channels - c0) / P.cpg, g0 = c0 / P.cpg;
  join_channels(ch, groups, P.cpg, (float)len,
                [&](int g, Mom m) { own[g] = make_float4((float)len * (float)P.cpg, m.mean, m.low, m.M); });
  cluster_arrive();
  cluster_wait();
  for (int g = threadIdx.x; g < groups; g += kThreads) {
    float4 e[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      e[r] = r < P.splits ? ld_cluster_f4(cluster_map(own + g, r)) : make_float4(0.f, 0.f, 0.f, 0.f);
    Joint J{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) J.take(e[r]);
    const float mean = J.rounded_mean(), rstd = rstd_of(J.M / J.n, P.eps);
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
    const int64_t ystep = at.step * P.os[1];
#pragma unroll 4
    for (int i = 0; i < at.count; ++i) {
      float v[V];
      unpack<T, V>(load_raw<T, V>(mine + i * (kThreads * V)), v);
      f.z(v);
      activate<T>(v, P.act);
      store_f32<T, V>(y, v);
      y += ystep;
    }
  }
  cluster_wait();  // a block's memory stays until every peer has read it
}

// ---------------------------------------------------------------- gradient
// dz of one run and xm = x - mean; B sums dz xm, and takes its rstd at the end.
template <typename T, int V>
DIT_DEV void dz_of(const Affine<V>& f, const float (&x)[V], const float (&dy)[V], int act, float (&xm)[V], float (&dz)[V]) {
  v_sub(xm, x, f.mean);
  if (act == DIT_ACT_SILU) {
    float z[V], s[V], t[V];
    v_fma(z, xm, f.scale, f.bias);
    v_sigmoid<T>(s, t, z);
    v_fma(s, z, t, s);
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
// Sums of a thread; of few channels in two levels of 16 pixels, since the sums of
// few channels are many pixels long and may cancel.
template <int V>
struct GradSums {
  float A[V], B[V], a[V], b[V];
  int n;
  DIT_DEV GradSums() : n(0) { v_set(A, 0.f), v_set(B, 0.f), v_set(a, 0.f), v_set(b, 0.f); }
  DIT_DEV void add(const float (&dz)[V], const float (&xm)[V]) {
    if constexpr (V < 4) {
      v_add(a, a, dz);
      v_fma(b, dz, xm, b);
      if ((++n & 15) == 0) fold();
    } else {
      v_add(A, A, dz);
      v_fma(B, dz, xm, B);
    }
  }
  DIT_DEV void fold() {
    v_add(A, A, a);
    v_add(B, B, b);
    v_set(a, 0.f), v_set(b, 0.f);
  }
};

// part[b, split, c] = (sum dz, sum dz xhat) over the split's pixels.  Shared
// memory: the ring, then sums [rows][slab * V + 1].
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, stream_blocks(V * sizeof(T)) < 4 ? stream_blocks(V * sizeof(T)) : 4) gn_grad_sums_kernel(const __grid_constant__ GnParams P) {
  extern __shared__ float4 raw_sm[];
  using F = Feed2<T, V, false>;
  float2* sm = reinterpret_cast<float2*>(reinterpret_cast<char*>(raw_sm) + F::kBytes);
  start_next();
  const uint32_t b = blockIdx.x / (uint32_t)P.splits, split = blockIdx.x - b * P.splits;
  const Place at(P, V, blockIdx.y, split, P.splits);
  F feed;
  feed.from(0, static_cast<const T*>(P.x) + b * P.xs[0] + at.p * P.xs[1] + at.c, at.step * P.xs[1]);
  feed.from(1, static_cast<const T*>(P.dy) + b * P.ds[0] + at.p * P.ds[1] + at.c, at.step * P.ds[1]);
  feed.start(raw_sm, at.count);
  const int width = P.slab * V;
  Affine<V> f;
  GradSums<V> S;
  if (at.on) {
    f.weights(P, at.c);
    f.statistics(at.c, P.cpg, [&](int g) { return make_float2(P.mean[(int64_t)b * P.groups + g], P.rstd[(int64_t)b * P.groups + g]); });
    feed.run([&](int, const Raw<T, V>(&r)[2]) {
      float v[V], g[V], xm[V], dz[V];
      unpack<T, V>(r[0], v);
      unpack<T, V>(r[1], g);
      dz_of<T>(f, v, g, P.act, xm, dz);
      S.add(dz, xm);
    });
    float r[V];
    spread(r, at.c, P.cpg, [&](int g) { return P.rstd[(int64_t)b * P.groups + g]; });
    if constexpr (V < 4) S.fold();
    v_mul(S.B, S.B, r);
  }
  const int c0 = blockIdx.y * width, here = min(width, P.channels - c0);
  float2* part = P.part + (int64_t)blockIdx.x * P.channels + c0;
  sum_rows<V>(at, S.A, S.B, sm, P.slab, P.part_lanes, [&](int c, float2 v) {
    if (c < here) part[c] = v;
  });
}

// Sums of `count` pairs at(i): in a row where they are few, else 128 in a row and those
// joined without loss, so that the sum of many is as good as that of 128.  (One wave's
// shares are at most 114 a thread: one more instruction for each pair of them made the
// gradient of 200000 x 256 with its short runs 5 us longer.)
template <class At>
DIT_DEV float2 long_sums(int count, At at) {
  auto some = [&](int from, int to) {
    float2 v = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int i = from; i < to; ++i) {
      const float2 e = at(i);
      v.x += e.x, v.y += e.y;
    }
    return v;
  };
  if (count <= 128) return some(0, count);
  LongSum x, y;
  for (int i = 0; i < count; i += 128) {
    const float2 v = some(i, min(count, i + 128));
    x.add(v.x), y.add(v.y);
  }
  return make_float2(x.value(), y.value());
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
  const uint32_t b = blockIdx.x / (uint32_t)P.groups;
  const int g = blockIdx.x - b * P.groups;
  const int rows = kThreads / cols, col = threadIdx.x % cols, row = threadIdx.x / cols;
  const float2* part = P.part + (int64_t)b * P.splits * P.channels + (int64_t)g * P.cpg;
  float s1 = 0.f, s2 = 0.f;
  wait_previous();
  for (int c0 = 0; c0 < P.cpg; c0 += cols) {
    float A = 0.f, B = 0.f;
    if (c0 + col < P.cpg) {
      const float2* mine = part + (int64_t)row * P.channels + c0 + col;
      const int64_t step = (int64_t)rows * P.channels;
      const float2 v = long_sums((P.splits - row + rows - 1) / rows, [&](int i) { return mine[i * step]; });
      A = v.x, B = v.y;
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
      P.chan[(int64_t)b * P.channels + c] = make_float2(A, B);
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
  const float2 v = long_sums((int)P.batch, [&](int b) { return P.chan[(int64_t)b * P.channels + c]; });
  if (P.db) P.db[c] = v.x;
  if (P.dw) P.dw[c] = v.y;
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

// dx; the blocks behind the last share sum the channels over the batch.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, stream_blocks(V * sizeof(T)) < 4 ? stream_blocks(V * sizeof(T)) : 4) gn_grad_apply_kernel(const __grid_constant__ GnParams P) {
  extern __shared__ float4 raw_sm[];
  using F = Feed2<T, V, true>;
  const uint32_t work = (uint32_t)P.batch * P.passes;
  if (blockIdx.x >= work) {
    wait_previous();
    if (blockIdx.y == 0) grad_weights(P, (int)(blockIdx.x - work) * kThreads + threadIdx.x);
    return;
  }
  const uint32_t b = blockIdx.x / (uint32_t)P.passes, share = blockIdx.x - b * P.passes;
  const Place at(P, V, blockIdx.y, share, P.passes);
  // backwards, as gn_apply_kernel
  const int64_t last = at.p + (int64_t)(at.count - 1) * at.step, ostep = -at.step * P.os[1];
  F feed;
  feed.from(0, static_cast<const T*>(P.x) + b * P.xs[0] + last * P.xs[1] + at.c, -at.step * P.xs[1]);
  feed.from(1, static_cast<const T*>(P.dy) + b * P.ds[0] + last * P.ds[1] + at.c, -at.step * P.ds[1]);
  feed.start(raw_sm, at.count);
  Affine<V> f;
  GradApply<V> h;
  if (at.on) {
    f.weights(P, at.c);
    f.statistics(at.c, P.cpg, [&](int g) { return make_float2(P.mean[(int64_t)b * P.groups + g], P.rstd[(int64_t)b * P.groups + g]); });
  }
  wait_previous();
  if (!at.on) return;
  h.set(at.c, P.cpg, [&](int g) {
    const float2 s = P.gsum[(int64_t)b * P.groups + g];
    return make_float3(P.rstd[(int64_t)b * P.groups + g], s.x, s.y);
  });
  T* out = static_cast<T*>(P.out) + b * P.os[0] + last * P.os[1] + at.c;
  feed.run([&](int, const Raw<T, V>(&r)[2]) {
    float v[V], g[V], xm[V], dz[V];
    unpack<T, V>(r[0], v);
    unpack<T, V>(r[1], g);
    dz_of<T>(f, v, g, P.act, xm, dz);
    h.dx(f, xm, dz);
    store_f32_stream<T, V>(out, dz);
    out += ostep;
  });
}

// One launch, as gn_cluster_kernel: x and dy stay in shared memory between
// the sums and dx.  P.splits blocks take a batch element.  Where a cluster holds
// the whole batch's (P.whole_batch) it also joins the channel sums into dw and
// db; else a second launch does.
// Shared memory: sums [rows][slab * V + 1] float2, own [slab * V] float2 (read
// by the cluster), chan likewise, group sums [groups of the slab] float2, x, dy.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 2) gn_grad_cluster_kernel(const __grid_constant__ GnParams P, int data_elems) {
  extern __shared__ float4 raw_sm[];
  start_next();
  const int width = P.slab * V, rows = kThreads / (unsigned)P.slab, slab_groups = width / P.cpg;
  float2* sm = reinterpret_cast<float2*>(raw_sm);
  float2* own = sm + rows * (width + 1);
  float2* chan = own + width;
  float2* gs = chan + width;
  T* data = reinterpret_cast<T*>(raw_sm) +
            ((reinterpret_cast<char*>(gs + slab_groups) - reinterpret_cast<char*>(raw_sm) + 15) / 16 * 16) / sizeof(T);

  const uint32_t b = blockIdx.x / (uint32_t)P.splits;
  const int share = blockIdx.x - b * P.splits;
  const uint32_t base = cluster_ctarank() - share;  // rank of the batch element's first block
  const Place at(P, V, blockIdx.y, share, P.splits);
  const int c0 = blockIdx.y * width, here = min(width, P.channels - c0), groups = here / P.cpg, g0 = c0 / P.cpg;
  const float n = (float)P.pixels * (float)P.cpg;
  T* xs = data + threadIdx.x * V;
  T* gy = xs + data_elems;
  stage<T, V>(xs, static_cast<const T*>(P.x) + b * P.xs[0] + at.p * P.xs[1] + at.c, at.step * P.xs[1], at.count);
  stage<T, V>(gy, static_cast<const T*>(P.dy) + b * P.ds[0] + at.p * P.ds[1] + at.c, at.step * P.ds[1], at.count);
  const int64_t bg = (int64_t)b * P.groups;
  Affine<V> f;
  GradSums<V> S;
  if (at.on) {
    f.weights(P, at.c);
    f.statistics(at.c, P.cpg, [&](int g) { return make_float2(P.mean[bg + g], P.rstd[bg + g]); });
    staged();
#pragma unroll 2
    for (int i = 0; i < at.count; ++i) {
      float v[V], g[V], xm[V], dz[V];
      unpack<T, V>(load_raw<T, V>(xs + i * (kThreads * V)), v);
      unpack<T, V>(load_raw<T, V>(gy + i * (kThreads * V)), g);
      dz_of<T>(f, v, g, P.act, xm, dz);
      S.add(dz, xm);
    }
    float r[V];
    spread(r, at.c, P.cpg, [&](int g) { return P.rstd[bg + g]; });
    if constexpr (V < 4) S.fold();
    v_mul(S.B, S.B, r);
  }
  sum_rows<V>(at, S.A, S.B, sm, P.slab, P.part_lanes, [&](int c, float2 v) { own[c] = v; });
  cluster_arrive();
  cluster_wait();
  for (int c = threadIdx.x; c < here; c += kThreads) {
    LongSum x, y;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (r >= P.splits) continue;
      const float2 e = ld_cluster_f2(cluster_map(own + c, base + r));
      x.add(e.x), y.add(e.y);
    }
    const float A = x.value(), B = y.value();
    if (share == 0 && P.chan) P.chan[(int64_t)b * P.channels + c0 + c] = make_float2(A, B);
    const float w = P.w ? P.w[c0 + c] : 1.f;
    chan[c] = make_float2(w * A, w * B);
  }
  __syncthreads();
  if (P.whole_batch && blockIdx.x == 0) {
    // the batch's blocks in order
    for (int c = threadIdx.x; c < here; c += kThreads) {
      LongSum x, y;
      for (uint32_t r = 0; r < gridDim.x; ++r) {
        const float2 t = ld_cluster_f2(cluster_map(own + c, r));
        x.add(t.x), y.add(t.y);
      }
      if (P.db) P.db[c0 + c] = x.value();
      if (P.dw) P.dw[c0 + c] = y.value();
    }
  }
  cluster_arrive();  // this block has read its peers' memory
  if (P.cpg <= 8) {
    for (int g = threadIdx.x; g < groups; g += kThreads) {
      float s1 = 0.f, s2 = 0.f;
      for (int c = 0; c < P.cpg; ++c) s1 += chan[g * P.cpg + c].x, s2 += chan[g * P.cpg + c].y;
      gs[g] = make_float2(s1 / n, s2 / n);
    }
  } else {
    const int lane = threadIdx.x & 31;
    for (int g = threadIdx.x >> 5; g < groups; g += kThreads / 32) {
      float s1 = 0.f, s2 = 0.f;
      for (int c = lane; c < P.cpg; c += 32) s1 += chan[g * P.cpg + c].x, s2 += chan[g * P.cpg + c].y;
      s1 = warp_sum(s1), s2 = warp_sum(s2);
      if (lane == 0) gs[g] = make_float2(s1 / n, s2 / n);
    }
  }
  __syncthreads();
  if (at.on) {
    GradApply<V> h;
    h.set(at.c, P.cpg, [&](int g) { return make_float3(P.rstd[bg + g], gs[g - g0].x, gs[g - g0].y); });
    T* out = static_cast<T*>(P.out) + b * P.os[0] + at.p * P.os[1] + at.c;
    const int64_t ostep = at.step * P.os[1];
#pragma unroll 2
    for (int i = 0; i < at.count; ++i) {
      float v[V], g[V], xm[V], dz[V];
      unpack<T, V>(load_raw<T, V>(xs + i * (kThreads * V)), v);
      unpack<T, V>(load_raw<T, V>(gy + i * (kThreads * V)), g);
      dz_of<T>(f, v, g, P.act, xm, dz);
      h.dx(f, xm, dz);
      store_f32<T, V>(out, dz);
      out += ostep;
    }
  }
  cluster_wait();  // a block's memory stays until every peer has read it
}

// ---------------------------------------------------------------- plan
int elem_bytes(int dtype) { return dtype == DIT_DTYPE_F32 ? 4 : 2; }

bool aligned(const void* p, const int64_t st[2], int elem, int to) {
  return !p || (((uintptr_t)p | (uintptr_t)(st[0] * elem) | (uintptr_t)(st[1] * elem)) & (to - 1)) == 0;
}

// Channels a thread takes: 16, 8 or 4 bytes of them, or one.
int vec_of(const dit_group_norm_args& a) {
  const int e = elem_bytes(a.dtype);
  for (int to : {16, 8, 4})
    if (a.channels % (to / e) == 0 && aligned(a.x, a.x_stride, e, to) && aligned(a.dy, a.dy_stride, e, to) &&
        aligned(a.out, a.out_stride, e, to))
      return to / e;
  return 1;
}

struct Plan {
  bool cluster;
  int vec, slab, nslab, unit, splits, passes;
  bool fold;
  bool whole_batch;  // cluster form of the gradient, see GnParams
  int data_elems;  // cluster form: elements of one staged tensor
  size_t smem;
};

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr int64_t kSmemMost = 200 << 10;

size_t scratch_bytes(const Plan& p, int cpg, bool backward) {
  const int rows = kThreads / p.slab, width = p.slab * p.vec;
  size_t n = (size_t)rows * (width + 1) * 8;                          // sums
  if (!backward) n += (size_t)width * (sizeof(Mom) + sizeof(float));  // ch, piv
  if (p.cluster) n += backward ? (size_t)width * 16 + (size_t)(width / cpg) * 8 : (size_t)(width / cpg) * 24;
  return (n + 15) / 16 * 16;
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
  // shares of a batch element: one wave of blocks, fewer where a thread would
  // have less than four pixels, more where it would sum over too many in a row
  // for fp32
  const int64_t each = a.batch * p.nslab, most = a.pixels / ((int64_t)rows * 4);
  auto shares = [&](int blocks, int64_t least) {
    int64_t n = blocks / each;
    if (n > most) n = most;
    if (n < least) n = least;
    return (int)(n < 1 ? 1 : n);
  };
  const int wave = 152 * stream_blocks(vec * elem_bytes(a.dtype));
  p.splits = shares(wave, ceil_div(a.pixels, (int64_t)rows * (backward ? 128 : 256)));
  p.passes = shares(wave, 1);
  // few enough partials that every block of the pass joins its groups' itself
  p.fold = p.unit == cpg && (int64_t)p.splits * (p.slab * vec / cpg) <= 2048;
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
  p.splits = blocks;  // a cluster's last blocks may have no pixels
  p.unit = a.channels / a.groups;
  const int rows = kThreads / slab;
  const int64_t iters = ceil_div(a.pixels, (int64_t)blocks * rows);
  const int64_t data = iters * kThreads * vec * elem_bytes(a.dtype);
  if (data > kSmemMost) return p;
  const size_t smem = scratch_bytes(p, p.unit, backward) + (size_t)data * (backward ? 2 : 1);
  if (smem > (size_t)kSmemMost) return p;
  p.data_elems = (int)(iters * kThreads * vec);
  p.smem = smem;
  return p;
}

// The one-launch form where its blocks have little to do each: slabs of whole
// groups, at least 32 bytes of a pixel, no more of them than fill the SMs twice;
// pixels cut over a cluster until a thread has two (one wave) or eight of them
// (two waves).  Measured (bf16, us, one launch / three): 64 pixels x 320
// channels 5.1 / 7.7, 2 x 256 x 512 5.7 / 7.7, 4096 x 512 8.6 / 11.1, 8 x 1024 x
// 320 8.6 / 11.6, 4096 x 1024 10.4 / 13.5; with 16 pixels a thread 16384 x 128
// 10.1 / 9.3, 16 x 4096 x 128 13.4 / 13.0.  Gradient: 64 x 320 5.8 / 9.0, 4096 x
// 512 11.1 / 12.3, 4096 x 1024 13.4 / 18.5; where the weight sums of a batch
// take a second launch, 32 x 64 x 1280 at six pixels 13.1 / 16.2, 4 x 4096 x 256 at
// eight 15.6 / 14.6, so six is the limit there.
Plan plan_of(const dit_group_norm_args& a, int vec, bool backward) {
  const int cpg = a.channels / a.groups, runs = a.channels / vec, whole = cpg / gcd(cpg, vec);
  const int run_bytes = vec * elem_bytes(a.dtype);
  if (a.pixels && whole <= kThreads) {
    int slab = whole;
    auto slabs = [&] { return a.batch * ceil_div(runs, slab); };
    while (2 * slab <= kThreads && slab < runs && (slab * run_bytes < 32 || slabs() > 304)) slab *= 2;
    int blocks = 1;
    auto pixels = [&] { return ceil_div(a.pixels, (int64_t)blocks * (kThreads / slab)); };
    while (blocks < kMaxCluster && ((pixels() > 2 && 2 * blocks * slabs() <= 152) || (pixels() > 8 && 2 * blocks * slabs() <= 304)))
      blocks *= 2;
    const bool whole_batch = backward && a.batch * blocks <= kMaxCluster;
    if (blocks * slabs() <= 304 && pixels() <= (backward && !whole_batch ? 6 : 8)) {
      Plan p = cluster_plan(a, vec, slab, blocks, backward);
      p.whole_batch = whole_batch;
      if (p.smem) return p;
    }
  }
  return split_plan(a, vec, backward);
}

int64_t round256(int64_t n) { return (n + 255) & ~(int64_t)255; }

// Workspace of a plan: partials, then [batch, groups] pairs, then channel sums.
int64_t part_bytes(const dit_group_norm_args& a, const Plan& p, bool backward) {
  return p.cluster ? 0 : round256(a.batch * p.splits * (int64_t)(a.channels / p.unit) * (backward ? 8 : 16));
}
int64_t group_bytes(const dit_group_norm_args& a, const Plan& p) { return p.cluster ? 0 : round256(a.batch * a.groups * 8); }
int64_t chan_bytes(const dit_group_norm_args& a, const Plan& p, bool backward) {
  return !backward || p.whole_batch ? 0 : round256(a.batch * (int64_t)a.channels * 8);
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
    GN_TRY(launch_kernel(gn_grad_cluster_kernel<T, V>, grid, kThreads, pl.smem, s, pl.whole_batch ? (int)grid.x : pl.splits, false,
                         P, pl.data_elems));
    return extra && !pl.whole_batch ? launch_kernel(gn_grad_weights_kernel, dim3(extra), kThreads, 0, s, 1, true, P) : cudaSuccess;
  }
  const size_t ring = Feed1<T, V, false>::kBytes, ring2 = Feed2<T, V, false>::kBytes;
  if (!backward) {
    GN_TRY(launch_kernel(gn_sums_kernel<T, V>, grid, kThreads, ring + pl.smem, s, 1, false, P));
    if (!pl.fold) GN_TRY(launch_kernel(gn_join_kernel, bg, kJoinThreads, 0, s, 1, true, P));
    return launch_kernel(gn_apply_kernel<T, V>, pass, kThreads, ring + (pl.fold ? (size_t)pl.slab * V / P.cpg * 8 : 0), s, 1, true, P);
  }
  int cols = 1;
  while (cols < P.cpg && cols < 32) cols *= 2;
  GN_TRY(launch_kernel(gn_grad_sums_kernel<T, V>, grid, kThreads, ring2 + pl.smem, s, 1, false, P));
  GN_TRY(launch_kernel(gn_grad_join_kernel, bg, kThreads, 0, s, 1, true, P, cols));
  return launch_kernel(gn_grad_apply_kernel<T, V>, dim3(pass.x + extra, pass.y), kThreads, ring2, s, 1, true, P);
}

template <typename T>
cudaError_t run_vec(const dit_group_norm_args& a, const Plan& pl, const GnParams& P, bool backward, cudaStream_t s) {
  constexpr int most = 16 / sizeof(T);
  if (pl.vec == most) return run<T, most>(a, pl, P, backward, s);
  if (pl.vec == most / 2) return run<T, most / 2>(a, pl, P, backward, s);
  if constexpr (sizeof(T) == 2)
    if (pl.vec == 2) return run<T, 2>(a, pl, P, backward, s);
  return run<T, 1>(a, pl, P, backward, s);
}

}  // namespace

int64_t group_norm_workspace(const dit_group_norm_args& a, bool backward) {
  if (a.batch == 0) return 0;
  // enough for any alignment of the tensors
  int64_t need = 0;
  for (int vec : {16 / elem_bytes(a.dtype), 8 / elem_bytes(a.dtype), 4 / elem_bytes(a.dtype), 1}) {
    if (a.channels % vec) continue;
    const Plan p = plan_of(a, vec, backward);
    const int64_t n = part_bytes(a, p, backward) + group_bytes(a, p) + chan_bytes(a, p, backward);
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
  P.pixels = (int)a.pixels;
  P.channels = a.channels;
  P.groups = a.groups;
  P.cpg = a.channels / a.groups;
  P.splits = pl.splits;
  P.passes = pl.passes;
  P.slab = pl.slab;
  for (P.part_lanes = 1; P.part_lanes < 32 && 2 * P.part_lanes * pl.slab * pl.vec <= kThreads; P.part_lanes *= 2) {}
  P.unit = pl.unit;
  P.whole_batch = pl.whole_batch;
  P.fold = pl.fold;
  P.act = a.act;
  P.eps = a.eps;
  P.w = a.weight;
  P.b = a.bias;
  P.dw = a.dweight;
  P.db = a.dbias;
  char* ws = reinterpret_cast<char*>(workspace);
  P.sums = reinterpret_cast<float4*>(ws);
  P.part = reinterpret_cast<float2*>(ws);
  ws += part_bytes(a, pl, backward);
  float* bg = reinterpret_cast<float*>(ws);
  ws += group_bytes(a, pl);
  if (!backward) {
    P.mean_out = a.mean;
    P.rstd_out = a.rstd;
    if (!pl.cluster && !pl.fold) {
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
