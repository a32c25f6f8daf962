// Rotary position embedding of q and k by positions with several axes, with an
// optional RMS norm of every head in front of it, and the gradient of both.
//
// Mathematics.  Pair p of a head (channels (2p, 2p + 1) or (p, p + R/2)) of a
// token at position pos[a] turns by the angle pos[a] * theta^(-2j/axes[a]).
// The frequency is held in turns as a 64-bit fraction f, so the angle modulo
// one turn is the low 64 bits of the integer product pos * f: the reduction is
// exact however far the position (the only error is f's own, 2^-53 of it).
// The top two bits pick the quadrant and the remaining +-1/8 turn goes to
// sincospif.  With a norm: xhat = x r, r = (mean x^2 + eps)^-1/2, z = xhat w,
// y = R z.  Gradient: g = R^T dy; dw = sum g xhat; with h = g w,
// dx = r (h - xhat mean(h xhat)); the two row sums (x^2 and h x) are taken
// together, so a row costs one round of shuffles either way.
//
// What bounds it: HBM.  Every row is read once and written once.  A group of
// 4 to 32 lanes holds one row in registers (8 channels or more a lane, 128-bit
// accesses), keeps its pairs' cos and sin for all the heads of a slice, and
// has several rows' loads in flight.
#include <math.h>

#include "operators.h"
#include "vec.cuh"

namespace dit {

namespace {

constexpr int kRopeThreads = 256;

// ---------------------------------------------------------------- angles
// cos and sin of u / 2^64 turns.
DIT_DEV void turns_sincos(uint64_t u, float& c, float& s) {
  const uint32_t hi = (uint32_t)(u >> 32);
  const uint32_t k = (hi + 0x20000000u) >> 30;             // nearest quarter turn, 0..3
  const int32_t rem = (int32_t)(hi - (k << 30));           // in units of 2^-32 turns, |rem| <= 2^29
  float sr, cr;
  sincospif((float)rem * 4.656612873077393e-10f, &sr, &cr);  // 2^-31: half turns
  const float a = (k & 1) ? sr : cr, b = (k & 1) ? cr : sr;  // quarter turns swap and negate
  c = (k == 1 || k == 2) ? -a : a;
  s = (k >= 2) ? -b : b;
}
// Low 64 bits of position * f for an fp32 position m * 2^e: the 88-bit
// product of its 24-bit magnitude with f, shifted by e.
DIT_DEV uint64_t turns_of(float pos, uint64_t f) {
  const uint32_t bits = __float_as_uint(pos);
  const int be = (bits >> 23) & 255;
  const uint64_t m = (bits & 0x7FFFFFu) | (be ? 0x800000u : 0u);
  const int e = (be ? be : 1) - 150;
  const uint64_t lo = m * f, hi = __umul64hi(m, f);
  uint64_t u;
  if (e >= 64 || e <= -128) u = 0;
  else if (e >= 0) u = lo << e;
  else if (e > -64) u = (lo >> -e) | (hi << (64 + e));
  else u = hi >> (-e - 64);
  return (bits >> 31) ? 0 - u : u;
}
DIT_DEV bool finite_bits(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

// ---------------------------------------------------------------- row layouts
// A layout says which channels of a row a lane holds: NP pairs (a[i], b[i]).
// Pairs from R/2 on are pairs of channels that are not turned.

// Interleaved pairs, one run of 8 channels a lane.
template <typename T>
struct Interleaved8 {
  using Elem = T;
  static constexpr int NP = 4;
  struct RowRaw {
    Raw<T, 8> c;
  };
  int lane, slots;
  DIT_DEV void init(int lane_, int d, int, int) {
    lane = lane_;
    slots = d / 8;
  }
  DIT_DEV int pair(int i) const { return 4 * lane + i; }
  DIT_DEV bool has(int) const { return lane < slots; }
  DIT_DEV int chan_a(int i) const { return 8 * lane + 2 * i; }
  DIT_DEV int chan_b(int i) const { return 8 * lane + 2 * i + 1; }
  DIT_DEV bool has_b(int) const { return lane < slots; }
  DIT_DEV void load(RowRaw& r, const T* row, bool ok) const {
    r.c = ok && lane < slots ? load_raw<T, 8>(row + 8 * lane) : zero_raw<T, 8>();
  }
  DIT_DEV void values(const RowRaw& r, float (&a)[NP], float (&b)[NP]) const {
    float f[8];
    unpack<T, 8>(r.c, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = f[2 * i], b[i] = f[2 * i + 1];
  }
  DIT_DEV void store(T* row, const float (&a)[NP], const float (&b)[NP]) const {
    if (lane >= slots) return;
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = a[i], f[2 * i + 1] = b[i];
    store_f32<T, 8>(row + 8 * lane, f);
  }
};

// Split pairs, V channels of each half a lane (R/2 and head_dim multiples of
// V); the channels behind R in runs of 2 V, the last of which may be V.
template <typename T, int V>
struct SplitV {
  using Elem = T;
  static constexpr int NP = V;
  struct RowRaw {
    Raw<T, V> c0, c1;
  };
  int o0, o1, first;
  bool on0, on1;
  DIT_DEV void init(int lane, int d, int half, int) {
    const int turned = half / V;
    const int u = lane - turned;
    o0 = u < 0 ? lane * V : 2 * half + 2 * V * u;
    o1 = u < 0 ? half + lane * V : o0 + V;
    on0 = o0 < d;
    on1 = o1 < d;
    first = lane * V;
  }
  DIT_DEV int pair(int i) const { return first + i; }
  DIT_DEV bool has(int) const { return on0; }
  DIT_DEV bool has_b(int) const { return on1; }
  DIT_DEV int chan_a(int i) const { return o0 + i; }
  DIT_DEV int chan_b(int i) const { return o1 + i; }
  DIT_DEV void load(RowRaw& r, const T* row, bool ok) const {
    r.c0 = ok && on0 ? load_raw<T, V>(row + o0) : zero_raw<T, V>();
    r.c1 = ok && on1 ? load_raw<T, V>(row + o1) : zero_raw<T, V>();
  }
  DIT_DEV void values(const RowRaw& r, float (&a)[NP], float (&b)[NP]) const {
    unpack<T, V>(r.c0, a);
    unpack<T, V>(r.c1, b);
  }
  DIT_DEV void store(T* row, const float (&a)[NP], const float (&b)[NP]) const {
    if (on0) store_f32<T, V>(row + o0, a);
    if (on1) store_f32<T, V>(row + o1, b);
  }
};

// Any style, width, stride and alignment: a warp a row, pairs lane + 32 i,
// element accesses.
template <typename T, int N>
struct AnyPairs {
  using Elem = T;
  static constexpr int NP = N;
  struct RowRaw {
    T a[NP], b[NP];
  };
  int lane, pairs, half, split;
  DIT_DEV void init(int lane_, int d, int half_, int split_) {
    lane = lane_;
    pairs = d / 2;
    half = half_;
    split = split_;
  }
  DIT_DEV int pair(int i) const { return lane + 32 * i; }
  DIT_DEV bool has(int i) const { return pair(i) < pairs; }
  DIT_DEV bool has_b(int i) const { return has(i); }
  DIT_DEV int chan_a(int i) const { return split && pair(i) < half ? pair(i) : 2 * pair(i); }
  DIT_DEV int chan_b(int i) const { return split && pair(i) < half ? pair(i) + half : 2 * pair(i) + 1; }
  DIT_DEV void load(RowRaw& r, const T* row, bool ok) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      r.a[i] = ok && has(i) ? row[chan_a(i)] : from_f32<T>(0.f);
      r.b[i] = ok && has(i) ? row[chan_b(i)] : from_f32<T>(0.f);
    }
  }
  DIT_DEV void values(const RowRaw& r, float (&a)[NP], float (&b)[NP]) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) a[i] = to_f32(r.a[i]), b[i] = to_f32(r.b[i]);
  }
  DIT_DEV void store(T* row, const float (&a)[NP], const float (&b)[NP]) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (!has(i)) continue;
      row[chan_a(i)] = from_f32<T>(a[i]);
      row[chan_b(i)] = from_f32<T>(b[i]);
    }
  }
};

// ---------------------------------------------------------------- the kernel
enum RopeMode { ROPE_TURN = 0, ROPE_NORM = 1, ROPE_NORM_GRAD = 2 };

struct RopeSeg {
  const void* x;
  const void* dy;
  void* out;
  int64_t xs[3], ds[3], os[3];
  const float* w;
  float* part;  // ROPE_NORM_GRAD: [blocks][head_dim] partial dweight, or NULL
  int heads;
};

struct RopeParams {
  RopeSeg seg[2];
  const void* pos;
  int64_t ps[2];
  uint32_t tokens, rows;  // rows = batch * tokens
  int d, half, n_axes, pos_f32, negate, split, group_log2;
  int ends[DIT_ROPE_MAX_AXES];  // last pair + 1 of each axis
  float eps, inv_d;
  uint64_t turn[DIT_ROPE_MAX_HEAD_DIM / 2];
};

// blockIdx.y of gridDim.y: a slice of q's heads and of k's; blockIdx.x strides
// over tokens.  A group of 2^group_log2 lanes takes one token at a time: its
// angles once, then the slice's heads HU at a time.  A row's turn is
// ya = a k0 + b k1, yb = a k2 + b k3 with (k0, k1, k2, k3) = (c, -s, s, c), or
// with the norm's weights in them, on column pairs (fma.rn.f32x2).
template <class L, int MODE, int HU>
__global__ void __launch_bounds__(kRopeThreads, MODE == ROPE_NORM_GRAD ? 2 : 3) rope_kernel(const __grid_constant__ RopeParams P) {
  using T = typename L::Elem;
  constexpr int NP = L::NP, N2 = NP / 2;
  const int lanes = 1 << P.group_log2;
  const int lane = threadIdx.x & (lanes - 1);
  const int groups = kRopeThreads >> P.group_log2;
  const int group = threadIdx.x >> P.group_log2;
  const bool partial = 2 * P.half < P.d;

  L lay;
  lay.init(lane, P.d, P.half, P.split);
  // every pair's frequency and axis
  __shared__ uint64_t turn[DIT_ROPE_MAX_HEAD_DIM / 2];
  __shared__ int axis[DIT_ROPE_MAX_HEAD_DIM / 2];
  if (threadIdx.x < P.half) {
    turn[threadIdx.x] = P.turn[threadIdx.x];
    int on = 0;
    for (int a = 0; a + 1 < P.n_axes; ++a) on += (int)threadIdx.x >= P.ends[a];
    axis[threadIdx.x] = on;
  }
  __syncthreads();
  bool turned[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) turned[i] = lay.has(i) && lay.pair(i) < P.half;
  float2 da[2][N2], db[2][N2];
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int i = 0; i < N2; ++i) da[g][i] = db[g][i] = make_float2(0.f, 0.f);

  const uint32_t step = gridDim.x * groups;
  // the loop runs while any group of the block has a row: lanes of a warp stay
  // together for the shuffles
  for (uint32_t base = blockIdx.x * groups; base < P.rows; base += step) {
    const uint32_t row = base + group;
    const bool ok = row < P.rows;
    const uint32_t b = ok ? row / P.tokens : 0, t = ok ? row - b * P.tokens : 0;
    float c[NP], s[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) c[i] = 1.f, s[i] = 0.f;
    if (ok) {
      const int64_t po = b * P.ps[0] + t * P.ps[1];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (!turned[i]) continue;
        const int p = lay.pair(i);
        if (P.pos_f32) {
          const float pos = static_cast<const float*>(P.pos)[po + axis[p]];
          turns_sincos(turns_of(pos, turn[p]), c[i], s[i]);
          if (!finite_bits(pos)) c[i] = s[i] = __int_as_float(0x7FFFFFFF);
        } else {
          const int32_t pos = static_cast<const int32_t*>(P.pos)[po + axis[p]];
          turns_sincos((uint64_t)(int64_t)pos * turn[p], c[i], s[i]);
        }
        if (P.negate) s[i] = -s[i];
      }
    }
#pragma unroll(MODE == ROPE_NORM_GRAD ? 2 : 1)  // the gradient's sums are registers of their own for q and k
    for (int g = 0; g < 2; ++g) {
      const RopeSeg& S = P.seg[g];
      const int h0 = S.heads * blockIdx.y / gridDim.y, h1 = S.heads * (blockIdx.y + 1) / gridDim.y;
      if (h0 >= h1) continue;
      float2 k0[N2], k1[N2], k2[N2], k3[N2], wa[N2], wb[N2];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        float va = 1.f, vb = 1.f;
        if constexpr (MODE != ROPE_TURN) {
          va = lay.has(i) ? S.w[lay.chan_a(i)] : 0.f;
          vb = lay.has_b(i) ? S.w[lay.chan_b(i)] : 0.f;
        }
        const float m0 = MODE == ROPE_NORM ? c[i] * va : c[i], m1 = MODE == ROPE_NORM ? -s[i] * vb : -s[i];
        const float m2 = MODE == ROPE_NORM ? s[i] * va : s[i], m3 = MODE == ROPE_NORM ? c[i] * vb : c[i];
        if (i & 1) k0[i / 2].y = m0, k1[i / 2].y = m1, k2[i / 2].y = m2, k3[i / 2].y = m3, wa[i / 2].y = va, wb[i / 2].y = vb;
        else k0[i / 2].x = m0, k1[i / 2].x = m1, k2[i / 2].x = m2, k3[i / 2].x = m3, wa[i / 2].x = va, wb[i / 2].x = vb;
      }
      const T* x = static_cast<const T*>(S.x) + b * S.xs[0] + t * S.xs[1] + h0 * S.xs[2];
      const T* dy = MODE == ROPE_NORM_GRAD ? static_cast<const T*>(S.dy) + b * S.ds[0] + t * S.ds[1] + h0 * S.ds[2] : nullptr;
      T* out = static_cast<T*>(S.out) + b * S.os[0] + t * S.os[1] + h0 * S.os[2];
      for (int h = h0; h < h1; h += HU) {
        typename L::RowRaw rx[HU], rg[MODE == ROPE_NORM_GRAD ? HU : 1];
#pragma unroll
        for (int u = 0; u < HU; ++u) {
          lay.load(rx[u], x + u * S.xs[2], ok && h + u < h1);
          if constexpr (MODE == ROPE_NORM_GRAD) lay.load(rg[u], dy + u * S.ds[2], ok && h + u < h1);
        }
#pragma unroll
        for (int u = 0; u < HU; ++u) {
          const bool on = ok && h + u < h1;
          float af[NP], bf[NP];
          float2 a[N2], e[N2], ya[N2], yb[N2];
          lay.values(rx[u], af, bf);
#pragma unroll
          for (int i = 0; i < N2; ++i) a[i] = make_float2(af[2 * i], af[2 * i + 1]), e[i] = make_float2(bf[2 * i], bf[2 * i + 1]);
          if constexpr (MODE != ROPE_NORM_GRAD) {
#pragma unroll
            for (int i = 0; i < N2; ++i) {
              ya[i] = ffma2(a[i], k0[i], fmul2(e[i], k1[i]));
              yb[i] = ffma2(a[i], k2[i], fmul2(e[i], k3[i]));
            }
            if (partial) {  // channels that are not turned do not meet their neighbours (0 * inf)
#pragma unroll
              for (int i = 0; i < N2; ++i) {
                if (!turned[2 * i]) ya[i].x = a[i].x * k0[i].x, yb[i].x = e[i].x * k3[i].x;
                if (!turned[2 * i + 1]) ya[i].y = a[i].y * k0[i].y, yb[i].y = e[i].y * k3[i].y;
              }
            }
            if constexpr (MODE == ROPE_NORM) {
              float2 q = fmul2(a[0], a[0]);
              q = ffma2(e[0], e[0], q);
#pragma unroll
              for (int i = 1; i < N2; ++i) q = ffma2(e[i], e[i], ffma2(a[i], a[i], q));
              float ss = q.x + q.y;
              for (int o = lanes >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
              const float r = rsqrtf(fmaf(ss, P.inv_d, P.eps));
              const float2 r2 = make_float2(r, r);
#pragma unroll
              for (int i = 0; i < N2; ++i) ya[i] = fmul2(ya[i], r2), yb[i] = fmul2(yb[i], r2);
            }
          } else {
            float gaf[NP], gbf[NP];
            float2 ga[N2], gb[N2], q = make_float2(0.f, 0.f), dt = make_float2(0.f, 0.f);
            lay.values(rg[u], gaf, gbf);
#pragma unroll
            for (int i = 0; i < N2; ++i) {
              const float2 va = make_float2(gaf[2 * i], gaf[2 * i + 1]), vb = make_float2(gbf[2 * i], gbf[2 * i + 1]);
              ga[i] = ffma2(va, k0[i], fmul2(vb, k2[i]));
              gb[i] = ffma2(va, k1[i], fmul2(vb, k3[i]));
              if (partial) {
                if (!turned[2 * i]) ga[i].x = va.x, gb[i].x = vb.x;
                if (!turned[2 * i + 1]) ga[i].y = va.y, gb[i].y = vb.y;
              }
              q = ffma2(e[i], e[i], ffma2(a[i], a[i], q));
              dt = ffma2(fmul2(ga[i], wa[i]), a[i], dt);
              dt = ffma2(fmul2(gb[i], wb[i]), e[i], dt);
            }
            float ss = q.x + q.y, dot = dt.x + dt.y;
            for (int o = lanes >> 1; o; o >>= 1) {
              ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
              dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
            }
            const float r = rsqrtf(fmaf(ss, P.inv_d, P.eps));
            const float m = -dot * r * r * P.inv_d;  // dx = r (g w) + x r m
            const float2 r2 = make_float2(r, r), m2 = make_float2(r * m, r * m);
            const float2 on2 = on ? r2 : make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < N2; ++i) {
              ya[i] = ffma2(a[i], m2, fmul2(fmul2(ga[i], wa[i]), r2));
              yb[i] = ffma2(e[i], m2, fmul2(fmul2(gb[i], wb[i]), r2));
              da[g][i] = ffma2(fmul2(ga[i], on2), a[i], da[g][i]);
              db[g][i] = ffma2(fmul2(gb[i], on2), e[i], db[g][i]);
            }
          }
          if (on) {
#pragma unroll
            for (int i = 0; i < N2; ++i) af[2 * i] = ya[i].x, af[2 * i + 1] = ya[i].y, bf[2 * i] = yb[i].x, bf[2 * i + 1] = yb[i].y;
            lay.store(out + u * S.os[2], af, bf);
          }
        }
        x += HU * S.xs[2];
        dy += HU * S.ds[2];
        out += HU * S.os[2];
      }
    }
  }

  if constexpr (MODE == ROPE_NORM_GRAD) {
    // the block's dweight: groups in order, through shared memory
    extern __shared__ float sm[];  // [groups][d]
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      if (!P.seg[g].part) continue;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (lay.has(i)) sm[group * P.d + lay.chan_a(i)] = i & 1 ? da[g][i / 2].y : da[g][i / 2].x;
        if (lay.has_b(i)) sm[group * P.d + lay.chan_b(i)] = i & 1 ? db[g][i / 2].y : db[g][i / 2].x;
      }
      __syncthreads();
      const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
      for (int ch = threadIdx.x; ch < P.d; ch += kRopeThreads) {
        float v = 0.f;
        for (int j = 0; j < groups; ++j) v += sm[j * P.d + ch];
        P.seg[g].part[block * P.d + ch] = v;
      }
    }
  }
}

// dweight[ch] = sum over blocks of the partials, in a fixed order: 32 channels
// a block, 32 warps taking every 32nd partial.
__global__ void __launch_bounds__(1024) rope_dweight_kernel(const float* p0, int n0, float* dw0, const float* p1,
                                                           int n1, float* dw1, int d) {
  __shared__ float sm[32][33];
  const float* p = blockIdx.y ? p1 : p0;
  float* dw = blockIdx.y ? dw1 : dw0;
  const int n = blockIdx.y ? n1 : n0;
  if (!dw) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ch = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (ch < d)
    for (int i = warp; i < n; i += 32) v += p[(int64_t)i * d + ch];
  sm[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && ch < d) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sm[i][lane];
    dw[ch] = v;
  }
}

// ---------------------------------------------------------------- launch
// How one tensor's rows are read: in runs of 8 (interleaved pairs) or twice 4
// channels (split pairs) a lane where the widths, strides and pointers are multiples of what those need,
// else element by element.
enum RopeLayout { LAYOUT_ANY = 0, LAYOUT_RUNS4 = 4, LAYOUT_RUNS8 = 8 };

bool aligned(const void* p, const int64_t st[3], int elem, int to) {
  return !p || (((uintptr_t)p | (uintptr_t)(st[0] * elem) | (uintptr_t)(st[1] * elem) | (uintptr_t)(st[2] * elem)) &
                (to - 1)) == 0;
}

int elem_bytes(int dtype) { return dtype == DIT_DTYPE_F32 ? 4 : 2; }

RopeLayout layout_of(const dit_rope_args& a, const dit_rope_heads& h, int half) {
  const int e = elem_bytes(a.dtype);
  auto ok = [&](int to) {
    return aligned(h.x, h.x_stride, e, to) && aligned(h.dy, h.dy_stride, e, to) && aligned(h.out, h.out_stride, e, to);
  };
  if (a.style == DIT_ROPE_INTERLEAVED) return a.head_dim % 8 == 0 && ok(16) ? LAYOUT_RUNS8 : LAYOUT_ANY;
  if (a.head_dim % 4 == 0 && half % 4 == 0 && ok(4 * e)) return LAYOUT_RUNS4;
  return LAYOUT_ANY;
}

int log2_ceil(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

template <class L, int MODE, int HU>
cudaError_t launch(const RopeParams& P, dim3 grid, cudaStream_t s) {
  const size_t sm = MODE == ROPE_NORM_GRAD ? (size_t)(kRopeThreads >> P.group_log2) * P.d * sizeof(float) : 0;
  rope_kernel<L, MODE, HU><<<grid, kRopeThreads, sm, s>>>(P);
  return cudaGetLastError();
}

// HU rows in flight a group: 64 bytes of each lane (element accesses: 2 rows)
template <class L, int HU>
cudaError_t launch_mode(const RopeParams& P, int mode, dim3 grid, cudaStream_t s) {
  if (mode == ROPE_TURN) return launch<L, ROPE_TURN, HU>(P, grid, s);
  if (mode == ROPE_NORM) return launch<L, ROPE_NORM, HU>(P, grid, s);
  return launch<L, ROPE_NORM_GRAD, HU / 2>(P, grid, s);
}

template <typename T>
cudaError_t launch_layout(const RopeParams& P, int layout, int mode, dim3 grid, cudaStream_t s) {
  if (layout == LAYOUT_RUNS4) return launch_mode<SplitV<T, 4>, 8 / sizeof(T)>(P, mode, grid, s);
  if (layout == LAYOUT_RUNS8) return launch_mode<Interleaved8<T>, 8 / sizeof(T)>(P, mode, grid, s);
  if (P.d <= 128) return launch_mode<AnyPairs<T, 2>, 2>(P, mode, grid, s);
  return launch_mode<AnyPairs<T, 4>, 2>(P, mode, grid, s);
}

}  // namespace

cudaError_t rope_run(const dit_rope_args& a, bool backward, float* workspace, cudaStream_t stream) {
  RopeParams P{};
  P.pos = a.pos;
  P.ps[0] = a.pos_stride[0];
  P.ps[1] = a.pos_stride[1];
  P.tokens = (uint32_t)a.tokens;
  P.rows = (uint32_t)(a.batch * a.tokens);
  P.d = a.head_dim;
  P.n_axes = a.n_axes;
  P.pos_f32 = a.pos_dtype == DIT_POS_F32;
  P.split = a.style == DIT_ROPE_SPLIT;
  P.eps = a.eps;
  P.inv_d = 1.f / (float)a.head_dim;
  for (int i = 0; i < a.n_axes; ++i) {
    for (int j = 0; j < a.axes[i] / 2; ++j)
      P.turn[P.half++] =
          (uint64_t)ldexp(pow((double)a.theta, -2.0 * j / a.axes[i]) * 0.15915494309189533577, 64);  // 1 / (2 pi)
    P.ends[i] = P.half;
  }

  const dit_rope_heads* h[2] = {&a.q, &a.k};
  int mode[2], layout[2], blocks[2] = {0, 0};
  float* part[2] = {workspace, nullptr};
  for (int i = 0; i < 2; ++i) {
    mode[i] = !h[i]->weight ? ROPE_TURN : backward ? ROPE_NORM_GRAD : ROPE_NORM;
    layout[i] = layout_of(a, *h[i], P.half);
  }
  if (P.rows) {
    // both segments in one launch where they run the same kernel
    const bool together = h[0]->heads && h[1]->heads && mode[0] == mode[1] && layout[0] == layout[1];
    for (int first = 0; first < 2; first += together ? 2 : 1) {
      const int last = together ? 1 : first;
      RopeParams Q = P;
      Q.group_log2 = 5;
      const int v = layout[first];
      if (v) Q.group_log2 = log2_ceil(P.split ? P.half / v + (P.d - 2 * P.half + 2 * v - 1) / (2 * v) : P.d / v);
      Q.negate = backward && mode[first] == ROPE_TURN;
      const int hmax = together && h[1]->heads > h[first]->heads ? h[1]->heads : h[first]->heads;
      if (!hmax) continue;
      for (int i = first; i <= last; ++i) {
        RopeSeg& S = Q.seg[i - first];
        const dit_rope_heads& H = *h[i];
        S.heads = H.heads;
        S.w = H.weight;
        const bool turn_grad = Q.negate;
        S.x = turn_grad ? H.dy : H.x;
        S.dy = H.dy;
        S.out = H.out;
        for (int k = 0; k < 3; ++k) {
          S.xs[k] = turn_grad ? H.dy_stride[k] : H.x_stride[k];
          S.ds[k] = H.dy_stride[k];
          S.os[k] = H.out_stride[k];
        }
      }
      // one slice of all heads shares the token's cos and sin best; as many as
      // it takes to give every SM four blocks otherwise
      int64_t nx = ((int64_t)P.rows + (kRopeThreads >> Q.group_log2) - 1) >> (8 - Q.group_log2);
      int64_t ny = (608 + nx - 1) / nx;
      if (ny > hmax) ny = hmax;
      if (ny > 256) ny = 256;
      if (mode[first] == ROPE_NORM_GRAD && nx * ny > kRopeGradBlocks / 2) nx = kRopeGradBlocks / 2 / ny;
      for (int i = first; i <= last; ++i)
        if (mode[i] == ROPE_NORM_GRAD && h[i]->dweight) {
          blocks[i] = (int)(nx * ny);
          if (i == 1) part[1] = part[0] + (int64_t)blocks[0] * P.d;
          Q.seg[i - first].part = part[i];
        }
      const dim3 grid((unsigned)nx, (unsigned)ny);
      cudaError_t e;
      if (a.dtype == DIT_DTYPE_F32) e = launch_layout<float>(Q, layout[first], mode[first], grid, stream);
      else if (a.dtype == DIT_DTYPE_BF16) e = launch_layout<__nv_bfloat16>(Q, layout[first], mode[first], grid, stream);
      else e = launch_layout<__half>(Q, layout[first], mode[first], grid, stream);
      if (e != cudaSuccess) return e;
    }
  }
  float* dw[2] = {backward ? a.q.dweight : nullptr, backward ? a.k.dweight : nullptr};
  if (dw[0] || dw[1]) {
    rope_dweight_kernel<<<dim3((P.d + 31) / 32, 2), 1024, 0, stream>>>(part[0], blocks[0], dw[0], part[1], blocks[1],
                                                                     dw[1], P.d);
    return cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace dit
