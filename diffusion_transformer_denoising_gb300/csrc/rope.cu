// Rotary position embedding of q and k by positions with several axes, with an
// optional RMS norm of every head in front of it, and the gradient of both.
//
// Mathematics.  Pair p of a head (channels (2p, 2p + 1) or (p, p + R/2)) of a
// token at position pos[a] turns by the angle pos[a] * theta^(-2j/axes[a]).
// The frequency is held in turns as a 64-bit fraction f, so the angle modulo
// one turn is the low 64 bits of the integer product pos * f: the reduction is
// exact however far the position.  What is left is f's own error, 2^-53 of it (1 /
// (2 pi) as a double holds it) and 2^-58: an angle a is off by |a| 2^-53 + |pos| 2^-55.
// The top two bits pick the quadrant and the remaining +-1/8 turn goes through
// two short polynomials.  With a norm: xhat = x r, r = (mean x^2 + eps)^-1/2, z = xhat w,
// y = R z.  Gradient: g = R^T dy; dw = sum g xhat; with h = g w,
// dx = r (h - xhat mean(h xhat)); the two row sums (x^2 and h x) are taken
// together, so a row costs one round of shuffles either way.
//
// What bounds it: HBM, once the latency is covered; with the norm, and more so
// for its gradient, the instructions of a row (0.65 and 0.61 of the issue slots).
// Every row is read once and written once.  A group of lanes holds one row in
// registers (8 channels a lane, 128-bit accesses), forms its pairs' cos and sin
// once for all the token's heads, and always has the next batch of rows (64 bytes
// a lane), of the next tensor or token too, and the next token's positions on
// their way.  Measured on one GB300 (bf16, 128-wide heads, 44/42/42): q and k of
// 2 x 32760 tokens x 12 heads 122 us = 6.59 TB/s (0.985 of the copy bandwidth);
// 32760 tokens with the norm, out of a packed projection, 68.9 us = 5.85 TB/s; its
// gradient 118.8 us = 5.09 TB/s (when it was 116: without the loads ahead 151 us,
// with the positions not among them 146 us).
#include <math.h>

#include <type_traits>

#include "launch.cuh"
#include "operators.h"
#include "vec.cuh"

namespace dit {

namespace {

constexpr int kRopeThreads = 256;

// ---------------------------------------------------------------- angles
// cos and sin of u / 2^64 turns.  The remaining angle x half turns, |x| <= 1/4,
// goes through the Taylor series of sin(pi x) and cos(pi x) about 0 (to x^9 and
// x^10: what is cut off is below 2^-28).  All 64 bits are in x, rounded twice, so
// small sines are as good as large ones: 6 x 2^-24 of themselves at most.  (One
// conversion of 64 bits took the video pair 122.0 us instead of 121.7, its gradient
// with the norm 118.8 instead of 118.0.)
DIT_DEV void turns_sincos(uint64_t u, float& c, float& s) {
  const uint32_t hi = (uint32_t)(u >> 32);
  const uint32_t k = (hi + 0x20000000u) >> 30;   // nearest quarter turn, 0..3
  const int32_t rem = (int32_t)(hi - (k << 30));  // in units of 2^-32 turns, |rem| <= 2^29
  const float x = fmaf((float)(uint32_t)u, 1.0842021724855044e-19f, (float)rem * 4.656612873077393e-10f);  // half turns
  const float q = x * x;
  float sr = fmaf(q, 0.08214588661112823f, -0.5992645293207921f);
  sr = fmaf(sr, q, 2.550164039877345f);
  sr = fmaf(sr, q, -5.16771278004997f);
  sr = fmaf(sr, q, 3.141592653589793f) * x;
  float cr = fmaf(q, -0.02580689139001406f, 0.23533063035889312f);
  cr = fmaf(cr, q, -1.3352627688545893f);
  cr = fmaf(cr, q, 4.058712126416768f);
  cr = fmaf(cr, q, -4.934802200544679f);
  cr = fmaf(cr, q, 1.f);
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
  float* dw;    // ROPE_NORM_GRAD on one cluster a tensor: dweight itself, or NULL
  int heads;
};

struct RopeParams {
  RopeSeg seg[2];
  const void* pos;
  int64_t ps[2];
  uint32_t tokens, rows;  // rows = batch * tokens
  int d, half, n_axes, pos_f32, negate, split, one_cluster;
  int slots;     // lanes of a row
  int per_warp;  // rows a warp takes side by side, where lanes reduce; else 0
  int ends[DIT_ROPE_MAX_AXES];  // last pair + 1 of each axis
  float eps, inv_d;
  uint64_t turn[DIT_ROPE_MAX_HEAD_DIM / 2];
};

// 4 bytes to shared memory in the background (zeros unless `some`), and the
// wait for all of the thread's.
DIT_DEV void cp_async4(void* dst, const void* src, bool some) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(some ? 4 : 0) : "memory");
}
DIT_DEV void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Pairs of values, one fp32 instruction each: the packed f32x2 forms took as long
// (video norm 70.5 us against 69.1) and more registers.
DIT_DEV float2 fma2(float2 a, float2 b, float2 c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }
DIT_DEV float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }

template <int N>
using Int = std::integral_constant<int, N>;

// Each of N values summed over the group's `slots` lanes, for all of them:
// lane l takes l + o while there is one, then all take the first lane's.  A power
// of two needs no last step, lanes taking their partners' both ways.
template <int N>
DIT_DEV void group_sums(float (&v)[N], int lane, int slots) {
  if ((slots & (slots - 1)) == 0) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      if (o >= slots) continue;
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] += __shfl_xor_sync(0xFFFFFFFFu, v[j], o);
    }
  } else {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      if (o >= slots) continue;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float t = __shfl_down_sync(0xFFFFFFFFu, v[j], o);
        if (lane + o < slots) v[j] += t;
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = __shfl_sync(0xFFFFFFFFu, v[j], (threadIdx.x & 31) - lane);
  }
}

// Two pairs turned; MIX: the first (tx) or second (ty) of them may be a pair of
// channels that are not turned (k1 = k2 = 0), which must not meet: 0 * inf.
template <bool MIX>
DIT_DEV void turn_pair(float2 a, float2 b, float2 k0, float2 k1, float2 k2, float2 k3, bool tx, bool ty, float2& ya,
                       float2& yb) {
  const float2 am = MIX ? make_float2(tx ? a.x : 0.f, ty ? a.y : 0.f) : a;
  const float2 bm = MIX ? make_float2(tx ? b.x : 0.f, ty ? b.y : 0.f) : b;
  ya = fma2(a, k0, mul2(bm, k1));
  yb = fma2(am, k2, mul2(b, k3));
}

// blockIdx.y of gridDim.y: a slice of q's heads and of k's; blockIdx.x strides
// over tokens.  A group of `slots` lanes takes one token at a time: its
// angles once, then the slice's heads in batches of HU rows, the next batch's
// loads (of the next tensor or token, too) in flight while one is worked on.
// A row's turn is ya = a k0 + b k1, yb = a k2 + b k3 with (k0, k1, k2, k3) =
// (c, -s, s, c), or with the norm's weights in them.
template <class L, int MODE, int HU>
__global__ void __launch_bounds__(kRopeThreads, MODE == ROPE_NORM_GRAD ? 2 : 3) rope_kernel(const __grid_constant__ RopeParams P) {
  using T = typename L::Elem;
  constexpr int NP = L::NP, N2 = NP / 2;
  constexpr bool GRAD = MODE == ROPE_NORM_GRAD;
  // groups lie back to back in the block, or where they reduce in each warp; the
  // lanes left over have no row
  const int in = MODE == ROPE_TURN ? threadIdx.x : threadIdx.x & 31;
  const int side = in / (unsigned)P.slots, lane = in - side * P.slots;
  const uint32_t groups = MODE == ROPE_TURN ? kRopeThreads / (unsigned)P.slots : kRopeThreads / 32 * P.per_warp;
  const bool spare = MODE == ROPE_TURN ? side >= (int)groups : side >= P.per_warp;
  const uint32_t group = MODE == ROPE_TURN ? side : threadIdx.x / 32 * P.per_warp + side;
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
  // each tensor's weights of the pairs (a, b), as the lanes hold them
  __shared__ float2 weight[MODE == ROPE_TURN ? 1 : 2][MODE == ROPE_TURN ? 1 : DIT_ROPE_MAX_HEAD_DIM / 2];
  if constexpr (MODE != ROPE_TURN) {
    if (!spare && group < 2 && P.seg[group].heads)
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (lay.has(i))
          weight[group][lay.pair(i)] = make_float2(P.seg[group].w[lay.chan_a(i)], lay.has_b(i) ? P.seg[group].w[lay.chan_b(i)] : 0.f);
  }
  __syncthreads();
  bool turned[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) turned[i] = lay.has(i) && lay.pair(i) < P.half;
  // the gradient's sums (a block takes one tensor only): of the last rows in
  // registers, of all before in shared memory, a pair of channels as (high, low)
  // twice, so that the sum of many rows is as good as that of kFoldRows
  constexpr int kFoldRows = 32;
  [[maybe_unused]] __shared__ float4 total[GRAD ? NP : 1][GRAD ? kRopeThreads : 1];
  [[maybe_unused]] int since = 0;
  float2 da[N2], db[N2];
#pragma unroll
  for (int i = 0; i < N2; ++i) da[i] = db[i] = make_float2(0.f, 0.f);
  if constexpr (GRAD)
#pragma unroll
    for (int i = 0; i < NP; ++i) total[i][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto fold = [&] {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float4 t = total[i][threadIdx.x];
      float low;
      t.x = two_sum(t.x, i & 1 ? da[i / 2].y : da[i / 2].x, low);
      t.y += low;
      t.z = two_sum(t.z, i & 1 ? db[i / 2].y : db[i / 2].x, low);
      t.w += low;
      total[i][threadIdx.x] = t;
    }
#pragma unroll
    for (int i = 0; i < N2; ++i) da[i] = db[i] = make_float2(0.f, 0.f);
    since = 0;
  };

  // the slice's heads of each tensor
  const auto first_head = [&](int g) { return (int)(P.seg[g].heads * blockIdx.y / gridDim.y); };
  const auto end_head = [&](int g) {
    return GRAD && g != blockIdx.z ? first_head(g) : (int)(P.seg[g].heads * (blockIdx.y + 1) / gridDim.y);
  };
  const int g_first = first_head(0) < end_head(0) ? 0 : 1, g_last = first_head(1) < end_head(1) ? 1 : 0;
  const uint32_t step = gridDim.x * groups;

  // the next batch: the block's token base, the tensor, its heads, its rows
  uint32_t base = blockIdx.x * groups, b, t;
  int g = g_first, h, h1;
  bool ok;
  const T* x;
  const T* dy = nullptr;
  T* out;
  // what a lane keeps for itself outside the registers: the next token's
  // position on every pair's axis (on its way), and the token's cos and sin
  __shared__ int32_t where[NP][kRopeThreads];
  __shared__ float2 spin[NP][kRopeThreads];
  auto token = [&] {
    ok = !spare && base + group < P.rows;
    b = ok ? (base + group) / P.tokens : 0;
    t = ok ? base + group - b * P.tokens : 0;
    const int32_t* pos = static_cast<const int32_t*>(P.pos) + b * P.ps[0] + t * P.ps[1];
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (turned[i]) cp_async4(&where[i][threadIdx.x], pos + axis[lay.pair(i)], ok);
  };
  auto tensor = [&] {
    const RopeSeg& S = P.seg[g];
    h = first_head(g);
    h1 = end_head(g);
    x = static_cast<const T*>(S.x) + b * S.xs[0] + t * S.xs[1] + h * S.xs[2];
    if constexpr (GRAD) dy = static_cast<const T*>(S.dy) + b * S.ds[0] + t * S.ds[1] + h * S.ds[2];
    out = static_cast<T*>(S.out) + b * S.os[0] + t * S.os[1] + h * S.os[2];
  };
  typename L::RowRaw rx[HU], rg[GRAD ? HU : 1];
  auto load = [&] {
#pragma unroll
    for (int u = 0; u < HU; ++u) {
      lay.load(rx[u], x, ok && h + u < h1);
      x += P.seg[g].xs[2];
      if constexpr (GRAD) {
        lay.load(rg[u], dy, ok && h + u < h1);
        dy += P.seg[g].ds[2];
      }
    }
  };

  float2 k0[N2], k1[N2], k2[N2], k3[N2], wa[N2], wb[N2];
  bool new_token = true, new_tensor = true;
  token();
  tensor();
  if (h < h1) load();
  else base = P.rows;
  // the loop runs while any group of the block has a row: lanes of a warp stay
  // together for the shuffles
  while (base < P.rows) {
    do {  // the gradient leaves after kFoldRows rows; an if around fold() in here cost 3 us of 120
      if (new_token) {
        cp_async_wait();
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          float c = 1.f, s = 0.f;
          if (turned[i]) {
            const uint64_t f = turn[lay.pair(i)];
            const int32_t at = where[i][threadIdx.x];
            if (P.pos_f32) {
              turns_sincos(turns_of(__int_as_float(at), f), c, s);
              if (!finite_bits(__int_as_float(at))) c = s = __int_as_float(0x7FFFFFFF);
            } else {
              turns_sincos((uint64_t)(int64_t)at * f, c, s);
            }
            if (P.negate) s = -s;
          }
          spin[i][threadIdx.x] = make_float2(c, s);
        }
      }
      if (new_tensor) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const float2 cs = spin[i][threadIdx.x];
          float va = 1.f, vb = 1.f;
          if constexpr (MODE != ROPE_TURN) {
            const float2 w = lay.has(i) ? weight[g][lay.pair(i)] : make_float2(0.f, 0.f);
            va = w.x, vb = w.y;
          }
          const float m0 = MODE == ROPE_NORM ? cs.x * va : cs.x, m1 = MODE == ROPE_NORM ? -cs.y * vb : -cs.y;
          const float m2 = MODE == ROPE_NORM ? cs.y * va : cs.y, m3 = MODE == ROPE_NORM ? cs.x * vb : cs.x;
          if (i & 1) k0[i / 2].y = m0, k1[i / 2].y = m1, k2[i / 2].y = m2, k3[i / 2].y = m3, wa[i / 2].y = va, wb[i / 2].y = vb;
          else k0[i / 2].x = m0, k1[i / 2].x = m1, k2[i / 2].x = m2, k3[i / 2].x = m3, wa[i / 2].x = va, wb[i / 2].x = vb;
        }
      }
      // this batch's rows out of the load registers, and the next batch's loads
      typename L::RowRaw cx[HU], cg[GRAD ? HU : 1];
#pragma unroll
      for (int u = 0; u < HU; ++u) {
        cx[u] = rx[u];
        if constexpr (GRAD) cg[u] = rg[u];
      }
      const bool row_ok = ok;
      T* const to = out;
      const int64_t to_step = P.seg[g].os[2];
      const int left = min(h1 - h, HU);
      h += HU;
      out += HU * to_step;
      new_tensor = new_token = false;
      if (h >= h1) {
        new_tensor = true;
        if (g == g_last) {
          new_token = true;
          base = P.rows - base > step ? base + step : P.rows;  // the sum can pass 2^32
          token();
          g = g_first;
        } else {
          g = 1;
        }
        tensor();
      }
      if (base < P.rows) load();
      // N rows of the batch at once, their chains of latency side by side; MIX:
      // some of the lane's channels are not turned
      auto rows = [&](auto first_, auto n_, auto mix_) {
        constexpr int N = decltype(n_)::value, first = decltype(first_)::value;
        constexpr bool MIX = decltype(mix_)::value;
        [[maybe_unused]] float2 a[N][N2], e[N][N2];
        float2 ya[N][N2], yb[N][N2];
        float ss[N], dot[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float af[NP], bf[NP];
          lay.values(cx[first + j], af, bf);
          float2 q = make_float2(0.f, 0.f), dt = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < N2; ++i) {
            const float2 va = make_float2(af[2 * i], af[2 * i + 1]), vb = make_float2(bf[2 * i], bf[2 * i + 1]);
            if constexpr (MODE != ROPE_TURN) q = fma2(vb, vb, fma2(va, va, q));
            if constexpr (GRAD) a[j][i] = va, e[j][i] = vb;
            else turn_pair<MIX>(va, vb, k0[i], k1[i], k2[i], k3[i], turned[2 * i], turned[2 * i + 1], ya[j][i], yb[j][i]);
          }
          if constexpr (GRAD) {
            lay.values(cg[first + j], af, bf);
#pragma unroll
            for (int i = 0; i < N2; ++i) {
              const float2 va = make_float2(af[2 * i], af[2 * i + 1]), vb = make_float2(bf[2 * i], bf[2 * i + 1]);
              turn_pair<MIX>(va, vb, k0[i], k2[i], k1[i], k3[i], turned[2 * i], turned[2 * i + 1], ya[j][i], yb[j][i]);
              dt = fma2(mul2(ya[j][i], wa[i]), a[j][i], dt);
              dt = fma2(mul2(yb[j][i], wb[i]), e[j][i], dt);
            }
          }
          ss[j] = q.x + q.y;
          dot[j] = dt.x + dt.y;
        }
        if constexpr (MODE != ROPE_TURN) {
          group_sums<N>(ss, lane, P.slots);
          if constexpr (GRAD) group_sums<N>(dot, lane, P.slots);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float r = rsqrtf(fmaf(ss[j], P.inv_d, P.eps));
            const float2 r2 = make_float2(r, r);
            if constexpr (!GRAD) {
#pragma unroll
              for (int i = 0; i < N2; ++i) ya[j][i] = mul2(ya[j][i], r2), yb[j][i] = mul2(yb[j][i], r2);
            } else {
              const float m = -dot[j] * r * r * r * P.inv_d;  // dx = r (g w) - x r^3 mean(g w x)
              const float2 m2 = make_float2(m, m);
#pragma unroll
              for (int i = 0; i < N2; ++i) {
                const float2 ga = mul2(ya[j][i], r2), gb = mul2(yb[j][i], r2);
                if (row_ok) da[i] = fma2(ga, a[j][i], da[i]), db[i] = fma2(gb, e[j][i], db[i]);
                ya[j][i] = fma2(a[j][i], m2, mul2(ga, wa[i]));
                yb[j][i] = fma2(e[j][i], m2, mul2(gb, wb[i]));
              }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float af[NP], bf[NP];
#pragma unroll
          for (int i = 0; i < N2; ++i)
            af[2 * i] = ya[j][i].x, af[2 * i + 1] = ya[j][i].y, bf[2 * i] = yb[j][i].x, bf[2 * i + 1] = yb[j][i].y;
          if (row_ok) lay.store(to + (first + j) * to_step, af, bf);
        }
      };
      // side by side only where two blocks an SM leave the registers for it
      constexpr int kSide = GRAD && HU > 1 ? 2 : 1;
      auto batch = [&](auto side_, auto mix, int n) {  // the first n rows, side_ at once
        constexpr int N = decltype(side_)::value;
        static_assert(HU <= 4 * N);
        rows(Int<0>{}, Int<N>{}, mix);
        if constexpr (HU >= 2 * N)
          if (n > N) rows(Int<N>{}, Int<N>{}, mix);
        if constexpr (HU >= 3 * N)
          if (n > 2 * N) rows(Int<2 * N>{}, Int<N>{}, mix);
        if constexpr (HU >= 4 * N)
          if (n > 3 * N) rows(Int<3 * N>{}, Int<N>{}, mix);
      };
      if (left < HU) batch(Int<1>{}, std::true_type{}, left);
      else if (partial) batch(Int<kSide>{}, std::true_type{}, HU);
      else batch(Int<kSide>{}, std::false_type{}, HU);
      since += left;
    } while (base < P.rows && (!GRAD || since < kFoldRows));
    if constexpr (GRAD) fold();
  }

  cp_async_wait();  // nothing of a token that never came is left on its way

  if constexpr (GRAD) {
    // the block's dweight: groups in order, through shared memory; then the
    // cluster's, where the tensor's blocks are one
    start_next();
    float *part = P.seg[blockIdx.z].part, *dw = P.seg[blockIdx.z].dw;
    extern __shared__ float sm[];  // [groups][d], then the block's [d]
    if (part || dw) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (spare) continue;
        const float4 t = total[i][threadIdx.x];
        if (lay.has(i)) sm[group * P.d + lay.chan_a(i)] = finite_bits(t.x) ? t.x + t.y : t.x;
        if (lay.has_b(i)) sm[group * P.d + lay.chan_b(i)] = finite_bits(t.z) ? t.z + t.w : t.z;
      }
      __syncthreads();
      const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
      float* own = sm + groups * P.d;
      for (int ch = threadIdx.x; ch < P.d; ch += kRopeThreads) {
        LongSum v;  // eight groups (there are 8 a row of a warp) as a tree, those without loss
        for (uint32_t j = 0; j < groups; j += 8) {
          float t[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) t[k] = sm[(j + k) * P.d + ch];
          v.add(((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7])));
        }
        if (part) part[block * P.d + ch] = v.value();
        else own[ch] = v.value();
      }
    }
    if (P.one_cluster) {
      cluster_arrive();
      cluster_wait();
      if (dw && blockIdx.x == 0)
        for (int ch = threadIdx.x; ch < P.d; ch += kRopeThreads) {
          LongSum v;
          for (uint32_t r = 0; r < gridDim.x; ++r) v.add(ld_cluster_f1(cluster_map(sm + groups * P.d + ch, r)));
          dw[ch] = v.value();
        }
      cluster_arrive();
      cluster_wait();  // a block's memory stays until it has been read
    }
  }
}

// dweight[ch] = sum over blocks of the partials, in a fixed order: 32 channels
// a block, 32 warps taking every 32nd partial, a warp joining a channel's.
__global__ void __launch_bounds__(1024) rope_dweight_kernel(const float* p0, int n0, float* dw0, const float* p1,
                                                           int n1, float* dw1, int d) {
  __shared__ float sm[32][33];
  const float* p = blockIdx.y ? p1 : p0;
  float* dw = blockIdx.y ? dw1 : dw0;
  const int n = blockIdx.y ? n1 : n0;
  if (!dw) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ch = blockIdx.x * 32 + lane;
  float v = 0.f;
  wait_previous();
  if (ch < d) {
#pragma unroll 4
    for (int i = warp; i < n; i += 32) v += p[(int64_t)i * d + ch];
  }
  sm[warp][lane] = v;
  __syncthreads();
  v = sm[lane][warp];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (lane == 0 && blockIdx.x * 32 + warp < d) dw[blockIdx.x * 32 + warp] = v;
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

template <class L, int MODE, int HU>
cudaError_t launch(const RopeParams& P, dim3 grid, cudaStream_t s) {
  const size_t sm = MODE == ROPE_NORM_GRAD ? (size_t)(kRopeThreads / 32 * P.per_warp + 1) * P.d * sizeof(float) : 0;
  return launch_kernel(rope_kernel<L, MODE, HU>, grid, dim3(kRopeThreads), sm, s, P.one_cluster ? (int)grid.x : 1, false, P);
}

// HU rows in flight a group: 64 bytes of each lane (element accesses: 2 rows)
template <class L, int HU>
cudaError_t launch_mode(const RopeParams& P, int mode, dim3 grid, cudaStream_t s) {
  if (mode == ROPE_TURN) return launch<L, ROPE_TURN, HU>(P, grid, s);
  if (mode == ROPE_NORM) return launch<L, ROPE_NORM, HU>(P, grid, s);
  return launch<L, ROPE_NORM_GRAD, (HU > 1 ? HU / 2 : 1)>(P, grid, s);
}

template <typename T>
cudaError_t launch_layout(const RopeParams& P, int layout, int mode, dim3 grid, cudaStream_t s) {
  if (layout == LAYOUT_RUNS4) return launch_mode<SplitV<T, 4>, 8 / sizeof(T)>(P, mode, grid, s);
  if (layout == LAYOUT_RUNS8) return launch_mode<Interleaved8<T>, 8 / sizeof(T)>(P, mode, grid, s);
  if (P.d <= 128) return launch_mode<AnyPairs<T, 2>, 2>(P, mode, grid, s);
  return launch_mode<AnyPairs<T, 4>, 2>(P, mode, grid, s);
}

// A value as the sum of two doubles, good to 2^-100 of it.
struct Twofold {
  double h, l;
};
Twofold operator*(Twofold a, Twofold b) {
  const double p = a.h * b.h, e = fma(a.h, b.h, -p) + (a.h * b.l + a.l * b.h), h = p + e;
  return {h, e - (h - p)};
}
// theta^(-1/m): pow's answer and one Newton step on r^m theta = 1.
Twofold root(float theta, int m) {
  const double r = pow((double)theta, -1.0 / m);
  Twofold p{theta, 0.0}, s{r, 0.0};
  for (int n = m; n; n >>= 1, s = s * s)
    if (n & 1) p = p * s;
  const double d = r * ((1.0 - p.h) - p.l) / m, h = r + d;
  return {h, d - (h - r)};
}
// r <= 1 in units of 2^-64, to the nearest (1 itself one unit less).
uint64_t fraction(Twofold r) {
  if (r.h >= 1.0) return UINT64_MAX;
  const double h = r.h * 0x1p64;
  const uint64_t i = (uint64_t)h;
  return i + (int64_t)floor((h - (double)i) + r.l * 0x1p64 + 0.5);
}

}  // namespace

// At most 12 turns of a cluster of eight blocks with eight groups each: there one
// launch takes as long as two (64 tokens x 3 heads 5.9 / 5.6 us, 256 x 3 8.1 /
// 5.9; 512 x 3 12.4 / 7.2) and needs no workspace.
bool rope_one_cluster(const dit_rope_args& a) {
  const int64_t rows = a.batch * a.tokens, heads = a.q.heads > a.k.heads ? a.q.heads : a.k.heads;
  return rows > 0 && (rows + 63) / 64 * heads <= 12;
}

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
    // powers of the neighbours' ratio in 64-bit fractions: half a unit of 2^-64 a step,
    // which shrink with the frequencies (128 pairs: below 64 units whatever theta)
    uint64_t f = (uint64_t)(0.15915494309189533577 * 0x1p64);  // 1 / (2 pi)
    const uint64_t r = a.axes[i] > 2 ? fraction(root(a.theta, a.axes[i] / 2)) : 0;
    for (int j = 0; j < a.axes[i] / 2; ++j) {
      P.turn[P.half++] = f;
      f = (uint64_t)(((unsigned __int128)f * r + (1ull << 63)) >> 64);
    }
    P.ends[i] = P.half;
  }

  const dit_rope_heads* h[2] = {&a.q, &a.k};
  int mode[2], layout[2], blocks[2] = {0, 0};
  float* part[2] = {workspace, workspace};
  bool joined[2] = {false, false};
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
      const int v = layout[first];
      Q.slots = !v ? 32 : P.split ? P.half / v + (P.d - 2 * P.half + 2 * v - 1) / (2 * v) : P.d / v;
      // lanes that reduce: a power of two unless the exact number lets a warp take
      // more rows (20000 tokens x 24 heads, gradient: 72 channels 58 against 69
      // us, but 96 channels 83 against 75, 160 channels 158 against 127)
      int wide = 1;
      while (wide < Q.slots) wide *= 2;
      if (mode[first] != ROPE_TURN && 32 / wide == 32 / Q.slots) Q.slots = wide;
      Q.per_warp = 32 / Q.slots;
      const int groups = mode[first] == ROPE_TURN ? kRopeThreads / Q.slots : kRopeThreads / 32 * Q.per_warp;
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
      const bool grad = mode[first] == ROPE_NORM_GRAD;
      const int nz = grad && together ? 2 : 1;
      int64_t nx = ((int64_t)P.rows + groups - 1) / groups;
      int64_t ny = (608 + nx * nz - 1) / (nx * nz);
      if (ny > hmax) ny = hmax;
      if (ny > 256) ny = 256;
      // the gradient keeps its weight sums in registers: as many blocks as run
      // at once, so few partials are left to join (two per SM: 115 us on the
      // 32760-token video gradient at the time, 127 us with 1024 blocks a tensor)
      if (grad && nx * ny > 304 / nz) nx = 304 / nz / ny > 0 ? 304 / nz / ny : 1;
      // few rows: a cluster of eight blocks a tensor joins the weight sums itself
      if (grad && rope_one_cluster(a) && (h[first]->dweight || h[last]->dweight)) {
        Q.one_cluster = 1;
        ny = 1;
        nx = kMaxCluster;
        for (int i = first; i <= last; ++i) {
          Q.seg[i - first].dw = h[i]->dweight;
          joined[i] = true;
        }
      }
      for (int i = first; i <= last; ++i)
        if (grad && h[i]->dweight && !joined[i]) {
          blocks[i] = (int)(nx * ny);
          if (i == 1) part[1] = part[0] + (int64_t)blocks[0] * P.d;
          Q.seg[i - first].part = part[i];
        }
      const dim3 grid((unsigned)nx, (unsigned)ny, (unsigned)nz);
      cudaError_t e;
      if (a.dtype == DIT_DTYPE_F32) e = launch_layout<float>(Q, layout[first], mode[first], grid, stream);
      else if (a.dtype == DIT_DTYPE_BF16) e = launch_layout<__nv_bfloat16>(Q, layout[first], mode[first], grid, stream);
      else e = launch_layout<__half>(Q, layout[first], mode[first], grid, stream);
      if (e != cudaSuccess) return e;
    }
  }
  float* dw[2] = {backward && !joined[0] ? a.q.dweight : nullptr, backward && !joined[1] ? a.k.dweight : nullptr};
  if (dw[0] || dw[1])
    return launch_kernel(rope_dweight_kernel, dim3((P.d + 31) / 32, 2), dim3(1024), 0, stream, 1, P.rows != 0, part[0],
                         blocks[0], dw[0], part[1], blocks[1], dw[1], P.d);
  return cudaSuccess;
}

}  // namespace dit
