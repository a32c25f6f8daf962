// Gated feed-forward: out = act(x Wg^T + bg) * (x Wu^T + bu), and its gradient.
//
// Mathematics.  M rows, width D, hidden F.  Forward: a tile's accumulator holds
// the gate's and the up projection's columns side by side, so the activation and
// the product happen as it leaves tensor memory.  With s = sigmoid(z), z = g (SiLU)
// or 2 c (g + 0.044715 g^3), c = sqrt(2 / pi) (GELU, tanh form: (1 + tanh u) / 2 =
// sigmoid(2 u)), act(g) = g s and act'(g) = s + g s (1 - s) z'.  Gradient: dU = dh act(g),
// dG = dh u act'(g) by an elementwise kernel that also sums the bias gradients;
// dx = dG Wg + dU Wu as one product over both halves of K; dWg = dG^T x and
// dWu = dU^T x as two products of one launch.
//
// All three products run on one persistent kernel: warp 0 loads operand tiles by
// TMA into a ring, warp 1 issues tcgen05.mma into one of two accumulators, eight
// warps drain the other.  What differs is which operand lies K-contiguous in
// memory: x and W rows in the forward, W rows across in dx, both operands across
// in dW.  Those tiles are loaded as they lie (64 channels x 64 K rows, 128-byte
// swizzle) and the MMA reads them MN-major, so nothing is transposed.
//
// What bounds it: the tensor cores, under the power cap in longer runs.  Measured on
// one GB300, 1536 x 8960 (device time of single launches): 32760 rows 940 to 960 us =
// 1.9 PFLOP/s (1090 us = 1.65 in a row of calls, 0.97 of the sustained peak); from
// e4m3 530 to 550 us = 3.3 PFLOP/s; gradient of 8190 rows: slopes 125 us (HBM), dx 261 us and dW
// 252 us = 1.75 PFLOP/s.  One row 10 us, 0.81 of the copy bandwidth.
//
// Measured slower: dx and dW as one launch, so that the tiles of one fill the last
// round of the other (568 us instead of 549 back to back: under the power cap idle SMs
// cost nothing, and the mix reads more from DRAM); tensor memory drained 16 columns
// at a time with the next ones on their way (e4m3 648 us, 578 at the time), or a
// whole unit at once (826 us, spilled); column groups narrower than the
// matrix (bf16 966 to 1057 us, 945 to 980 at the time).
#include <math.h>

#include "column_sums.cuh"
#include "common.cuh"
#include "launch.cuh"
#include "operators.h"
#include "tmap.h"
#include "vec.cuh"

namespace dit {

namespace {

// First site whose bounded wait ran out, 0: none (dit_gated_ffn_synchronize).
__device__ int g_wait_error;

enum Mode { FWD, DX, DW };

constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kSms = 152;  // the plan is made for this card, whatever device asks for it

// PAIR: 256 x 256 tiles on clusters of two CTAs (one tcgen05.mma.cta_group::2 of M
// = 256 a step; each CTA holds 128 rows of A and half of B's rows); else 128 x 128 on one.
template <bool F8, bool PAIR>
struct Cfg {
  static constexpr int BN = PAIR ? 256 : 128;  // accumulator columns
  static constexpr int BM = 128;               // accumulator rows of a CTA
  static constexpr int TILE_M = PAIR ? 256 : 128;
  static constexpr int BK = F8 ? 128 : 64;     // 128 bytes
  static constexpr int OPERAND = 128 * 128;    // bytes of a CTA's A or B tile
  static constexpr int STAGE = 2 * OPERAND;
  static constexpr int STAGES = 6;
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int STG_OFF = STAGES * STAGE;
  static constexpr int STG = 32 * 128;         // one warp's staging: 32 rows x 128 bytes
  static constexpr int BAR_OFF = STG_OFF + kEpiWarps * STG;
  static constexpr int SMEM = BAR_OFF + 256 + 1024;
  static constexpr int MMA_M = TILE_M;
};
static_assert(Cfg<false, true>::SMEM <= 232448, "tile set exceeds 227 KB of shared memory");

struct Product {
  CUtensorMap a[2], b[2], c[3];
  void* out[3];
  int64_t ldo[3];
  int tma[3];           // output by tensor stores; else by plain ones
  float* partial;       // splits > 1: fp32 planes [problem][split][gate, up][M][ldp]
  int64_t ldp, plane;
  const float *x_scale, *scale[2], *bias[2];
  int64_t M;            // rows and columns of the output
  int N;
  int k_blocks, k_half; // DX: blocks of each half of K
  int m_tiles, n_tiles, group_n, splits, items;
  int k_per;            // K blocks of a split; the last has the rest
  uint32_t idesc;
  int f16, act;
};

// ---------------------------------------------------------------- activation
// z = g (SiLU) or 2 sqrt(2 / pi) (g + 0.044715 g^3) (GELU, tanh form): act(g) = g sigmoid(z),
// by ex2.approx and rcp.approx.  The rounding of the exponent z log2 e counts most:
// 2^-16 of the value at |z| = 90, against the 2^-11 (fp16) of rounding it.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
DIT_DEV float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
DIT_DEV float fmin3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int ACT>
DIT_DEV float argument(float g) {
  return ACT == DIT_ACT_SILU ? g : g * fmaf(kGelu2 * 0.044715f, g * g, kGelu2);
}
// min(a, b), NaN if one of them is
DIT_DEV float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// sigmoid(z) and 1 - sigmoid(z), each on its own scale: subnormal numbers are kept.  Of
// NaN they are NaN and 0: GELU's slope takes sigmoid(z) alone where the other is 0.
DIT_DEV float2 sigmoids(float z) {
  const float m = min_nan(z * kLog2e, 126.f);
  float e;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(m));
  const float r = rcp_approx(1.f + e);
  return make_float2(e * r, m < 126.f ? r : 0.f);
}
// act(g) u of two columns.
template <int ACT>
DIT_DEV float2 gated2(float2 g, float2 u) {
  return make_float2(g.x * sigmoids(argument<ACT>(g.x)).x * u.x, g.y * sigmoids(argument<ACT>(g.y)).x * u.y);
}
// The same in fewer instructions for g above kFar, where 2^-z stays in range (below,
// sigmoid(z) would go to 0 too early: the result is g times it).
template <int ACT>
constexpr float kFar = ACT == DIT_ACT_SILU ? -80.f : -9.6f;
template <int ACT>
DIT_DEV float2 gated2_near(float2 g, float2 u) {
  float2 m;  // -z log2 e
  if constexpr (ACT == DIT_ACT_SILU) {
    m = fmul2(g, make_float2(-kLog2e, -kLog2e));
  } else {
    constexpr float k0 = -kGelu2 * kLog2e, k1 = k0 * 0.044715f;
    m = fmul2(g, ffma2(fmul2(g, g), make_float2(k1, k1), make_float2(k0, k0)));
  }
  const float2 d = fadd2(make_float2(ex2_approx(m.x), ex2_approx(m.y)), make_float2(1.f, 1.f));
  return fmul2(fmul2(g, make_float2(rcp_approx(d.x), rcp_approx(d.y))), u);
}
// act(g) and act'(g) = s + g s (1 - s) z'
template <int ACT>
DIT_DEV float2 activation_slope(float g) {
  const float2 s = sigmoids(argument<ACT>(g));
  const float gs = g * s.x;
  if constexpr (ACT == DIT_ACT_SILU) return make_float2(gs, fmaf(gs, s.y, s.x));
  // far out 1 - s is 0 and z' may be infinite: the limit of their product is 0
  const float zp = fmaf(3.f * 0.044715f * kGelu2, g * g, kGelu2);
  return make_float2(gs, s.y == 0.f || s.x == 0.f ? s.x : fmaf(gs * s.y, zp, s.x));
}

DIT_DEV uint32_t pack16(int f16, float lo, float hi) { return f16 ? pack2<__half>(lo, hi) : pack_bf16x2(lo, hi); }

// 32 values of a per-column array from column c on, `none` from n on or without an
// array.  One branch for all of them: with a branch for every four columns, which keeps
// the loads of a tile apart, the e4m3 video case took 728 us instead of 543.
DIT_DEV void columns32(float (&v)[32], const float* p, int c, int n, float none) {
  if (p && c + 32 <= n && ((reinterpret_cast<uintptr_t>(p + c) & 15) == 0)) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(p + c + j));
      v[j] = t.x, v[j + 1] = t.y, v[j + 2] = t.z, v[j + 3] = t.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = p && c + j < n ? __ldg(p + c + j) : none;
  }
}
// acc * scale * row_scale + bias over 32 columns.  The sum meets one scale, then the other:
// their product may vanish (a row's scale may be 2^-126) where the value does not.
template <bool SCALED>
DIT_DEV void finish32(float (&v)[32], const Product& P, int side, float row_scale, int c0) {
  float w[32];
  if constexpr (SCALED) {
    columns32(w, P.scale[side], c0, P.N, 0.f);
    const float2 rs = make_float2(row_scale, row_scale);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 x = fmul2(fmul2(make_float2(v[j], v[j + 1]), make_float2(w[j], w[j + 1])), rs);
      v[j] = x.x, v[j + 1] = x.y;
    }
  }
  if (P.bias[side]) {
    columns32(w, P.bias[side], c0, P.N, 0.f);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += w[j];
  }
}

// ---------------------------------------------------------------- tiles
struct Tile {
  int p, z, mb, nb;  // problem, split of K, row tile, column tile
};
// Items run problem by problem, split by split; within one, in column groups of
// group_n tiles, N-fastest (the group's B columns stay in L2 while A streams by).
DIT_DEV Tile tile_of(const Product& P, int item) {
  const int per = P.m_tiles * P.n_tiles;
  Tile t;
  const int pz = item / per;
  const int i = item - pz * per;
  t.p = pz / P.splits;
  t.z = pz - t.p * P.splits;
  const int group = P.m_tiles * P.group_n, g = i / group, in = i - g * group;
  const int width = min(P.group_n, P.n_tiles - g * P.group_n);
  t.mb = in / width;
  t.nb = g * P.group_n + in - t.mb * width;
  return t;
}

DIT_DEV void load32(uint32_t taddr, float (&v)[32]) { tmem_ld32(taddr, reinterpret_cast<uint32_t(&)[32]>(v)); }
DIT_DEV void wait32(float (&v)[32]) { tmem_ld_wait_regs(reinterpret_cast<uint32_t(&)[32]>(v)); }

// 32 values of the lane's row into half `hh` of the warp's staging unit (32 rows of
// 64 columns; 16-byte chunk j of row r at chunk j ^ (r % 8), as the tensor store reads it).
DIT_DEV void stage32(uint8_t* stg, int hh, int f16, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 w;
    w.x = pack16(f16, v[8 * j], v[8 * j + 1]);
    w.y = pack16(f16, v[8 * j + 2], v[8 * j + 3]);
    w.z = pack16(f16, v[8 * j + 4], v[8 * j + 5]);
    w.w = pack16(f16, v[8 * j + 6], v[8 * j + 7]);
    *reinterpret_cast<uint4*>(stg + lane * 128 + (((hh * 4 + j) ^ (lane & 7)) << 4)) = w;
  }
}
// The staging unit to columns col0.. of rows row0.. of output o.
DIT_DEV void store_unit(const Product& P, int o, uint8_t* stg, int64_t row0, int col0) {
  const int lane = threadIdx.x & 31;
  if (P.tma[o]) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(&P.c[o], stg, col0, (int)row0);
      bulk_commit();
    }
    return;
  }
  __syncwarp();
  // Rows of any alignment.
  uint16_t* out = static_cast<uint16_t*>(P.out[o]) + row0 * P.ldo[o] + col0;
  const int rows = (int)min((int64_t)32, P.M - row0);
  if (col0 + 64 <= P.N) {
    // Eight lanes a row: the aligned vectors inside the row's 128 bytes, each out of two
    // chunks; then the elements at its ends, eight lanes a row too: 16 stores a lane.
    const int k = lane & 7;
    auto chunk = [&](int r, int j) { return *reinterpret_cast<const uint4*>(stg + r * 128 + ((j ^ (r & 7)) << 4)); };
#pragma unroll 2
    for (int r = lane >> 3; r < rows; r += 4) {
      uint16_t* row = out + r * P.ldo[o];
      const int lead = (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / 2;  // elements before the first vector
      const uint4 v = chunk(r, k);
      if (lead == 0) {
        *reinterpret_cast<uint4*>(row + 8 * k) = v;
        continue;
      }
      if (k < 7) *reinterpret_cast<uint4*>(row + lead + 8 * k) = shift16(v, chunk(r, k + 1), 2 * lead);
      const int c = k < lead ? k : 56 + k;  // the ends' elements: [0, lead) and [lead + 56, 64)
      row[c] = *reinterpret_cast<const uint16_t*>(stg + r * 128 + (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2);
    }
  } else {
    const int c = 2 * lane;
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(stg + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
      uint16_t* at = out + r * P.ldo[o] + c;
      if (col0 + c < P.N) at[0] = (uint16_t)w;
      if (col0 + c + 1 < P.N) at[1] = (uint16_t)(w >> 16);
    }
  }
  __syncwarp();
}
DIT_DEV void staging_free() {  // the last tensor store has read the warp's staging unit
  if ((threadIdx.x & 31) == 0) bulk_wait_read0();
  __syncwarp();
}

// fp32 sums of the lane's row, 32 columns, to a plane of partial sums
DIT_DEV void store_partial(const Product& P, float* plane, int64_t row, int c0, const float (&v)[32]) {
  if (row >= P.M) return;
  float* at = plane + row * P.ldp + c0;
#pragma unroll
  for (int j = 0; j < 32; j += 4)
    if (c0 + j < P.N) *reinterpret_cast<float4*>(at + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);  // ldp is a multiple of 4
}

// One accumulator out of tensor memory: rows row0 .. row0 + 31 of this warp,
// units of 64 output columns half, half + 2, ...; release() after the last read.
template <int MODE, bool F8, int ACT, int BN, class Release>
DIT_DEV void drain(const Product& P, const Tile& t, uint32_t tacc, int64_t row0, int half, uint8_t* stg, Release release) {
  constexpr int COLS = MODE == FWD ? BN / 2 : BN;  // output columns of the tile
  const int lane = threadIdx.x & 31;
  const int64_t row = row0 + lane;
  auto done = [&]() {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) release();
  };
  if (half * 64 >= COLS) {
    done();
    return;
  }
  float row_scale = 1.f;
  if constexpr (MODE == FWD)
    if (P.x_scale && row < P.M) row_scale = __ldg(P.x_scale + row);
#pragma unroll 1
  for (int u = half; u * 64 < COLS; u += 2) {
    const bool last = (u + 2) * 64 >= COLS;
    const int col0 = t.nb * COLS + u * 64;
    if (P.splits > 1) {
      constexpr int SIDES = MODE == FWD ? 2 : 1;
#pragma unroll 1
      for (int i = 0; i < 2 * SIDES; ++i) {
        const int side = i >> 1, hh = i & 1;
        float v[32];
        load32(tacc + side * (BN / 2) + u * 64 + hh * 32, v);
        wait32(v);
        if (last && i == 2 * SIDES - 1) done();
        store_partial(P, P.partial + ((t.p * P.splits + t.z) * SIDES + side) * P.plane, row, col0 + hh * 32, v);
      }
      continue;
    }
    if constexpr (MODE == FWD) {
      // out, then gate and up where they are kept
#pragma unroll 1
      for (int o = P.out[1] ? 2 : 0; o >= 0; --o) {
        staging_free();
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh) {
          float g[32], v[32];
          const uint32_t at = tacc + u * 64 + hh * 32;
          if (o == 0) {
            load32(at, g);
            load32(at + BN / 2, v);
            wait32(g);
            wait32(v);
            if (last && hh == 1) done();
            finish32<F8>(g, P, 0, row_scale, col0 + hh * 32);
            finish32<F8>(v, P, 1, row_scale, col0 + hh * 32);
            float low = g[0];
#pragma unroll
            for (int j = 0; j < 32; j += 2) low = fmin3(low, g[j], g[j + 1]);
            if (__any_sync(0xffffffffu, low < kFar<ACT>)) {
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const float2 h = gated2<ACT>(make_float2(g[j], g[j + 1]), make_float2(v[j], v[j + 1]));
                v[j] = h.x, v[j + 1] = h.y;
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const float2 h = gated2_near<ACT>(make_float2(g[j], g[j + 1]), make_float2(v[j], v[j + 1]));
                v[j] = h.x, v[j + 1] = h.y;
              }
            }
          } else {
            load32(at + (o - 1) * (BN / 2), v);
            wait32(v);
            finish32<F8>(v, P, o - 1, row_scale, col0 + hh * 32);
          }
          stage32(stg, hh, P.f16, v);
        }
        if (col0 < P.N && row0 < P.M) store_unit(P, o, stg, row0, col0);
      }
    } else {
      staging_free();
#pragma unroll 1
      for (int hh = 0; hh < 2; ++hh) {
        float v[32];
        load32(tacc + u * 64 + hh * 32, v);
        wait32(v);
        if (last && hh == 1) done();
        stage32(stg, hh, P.f16, v);
      }
      if (col0 < P.N && row0 < P.M) store_unit(P, MODE == DW ? t.p : 0, stg, row0, col0);
    }
  }
}

template <int MODE, bool F8, bool PAIR, int ACT>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ Product P) {
  using C = Cfg<F8, PAIR>;
  constexpr bool A_MN = MODE == DW, B_MN = MODE != FWD;  // operands that lie across K
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drained = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* err = &g_wait_error;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // A pair's leader (rank 0) issues the MMAs of both CTAs; its full[] counts the
  // bytes of both CTAs' loads, its tempty[] the draining warps of both.
  const uint32_t rank = PAIR ? cluster_ctarank() : 0;
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&P.a[0]);
    tma_prefetch_desc(&P.b[0]);
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
    else tmem_alloc(tmem_slot, C::TMEM_COLS);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (PAIR) cluster_sync();  // both CTAs' barriers stand before any remote arrival or copy
  const uint32_t tmem_base = *tmem_slot;
  auto abort_pair = [&]() {
    if constexpr (PAIR) st_cluster_u32(cluster_map((const void*)abort_flag, rank ^ 1u), 1u);
  };
  wait_previous();  // operands that a kernel of the same call wrote
  start_next();
  const int first = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int stride = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer (one thread)
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      int issued[C::STAGES];
#pragma unroll
      for (int s = 0; s < C::STAGES; ++s) issued[s] = 0;
      bool ok = true;
      const uint32_t full_leader = PAIR ? cluster_map(full, 0) : 0;
      auto load = [&](uint8_t* dst, const CUtensorMap* m, int x, int y) {
        if constexpr (PAIR) tma_load_2d_pair(dst, m, full_leader + stage * (uint32_t)sizeof(uint64_t), x, y);
        else tma_load_2d(dst, m, &full[stage], x, y);
      };
      for (int item = first; ok && item < P.items; item += stride) {
        const Tile t = tile_of(P, item);
        const int a0 = PAIR ? (2 * t.mb + (int)rank) * C::BM : t.mb * C::BM;  // first row of A
        const int b0 = MODE == FWD ? t.nb * (C::BN / 2) : t.nb * C::BN + (int)rank * 128;
        const int kb0 = t.z * P.k_per, kb1 = min(P.k_blocks, kb0 + P.k_per);
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = mbar_wait(&empty[stage], phase ^ 1, abort_flag, err, 11);
          if (!ok) break;
          uint8_t* sa = smem + stage * C::STAGE;
          uint8_t* sb = sa + C::OPERAND;
          // the leader's arrival brings the bytes of both CTAs' loads
          if (leader) mbar_arrive_expect_tx(&full[stage], (PAIR ? 2 : 1) * C::STAGE);
          const int seg = MODE == DX && kb >= P.k_half ? 1 : 0;
          const int k0 = (kb - seg * P.k_half) * C::BK;
          if constexpr (A_MN) {
            load(sa, &P.a[t.p], a0, k0);
            load(sa + 8192, &P.a[t.p], a0 + 64, k0);
          } else {
            load(sa, &P.a[seg], k0, a0);
          }
          if constexpr (B_MN) {
            load(sb, &P.b[seg], b0, k0);
            load(sb + 8192, &P.b[seg], b0 + 64, k0);
          } else if constexpr (PAIR) {
            load(sb, &P.b[rank], k0, b0);  // rank 0 the gate's 128 channels, rank 1 the up projection's
          } else {
            load(sb, &P.b[0], k0, b0);     // 64 channels of each
            load(sb + 8192, &P.b[1], k0, b0);
          }
          ++issued[stage];
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) abort_pair();
      }
      if (!ok) {
        // wind down: every copy this thread started lands before the CTA exits
        volatile int no_abort = 0;
        if (leader) {
          for (int s = 0; s < C::STAGES; ++s)
            if (issued[s] > 0) mbar_wait(&full[s], (uint32_t)((issued[s] - 1) & 1), &no_abort, nullptr, 0);
        } else {
          // the peer's loads complete on the leader's barriers, which need the
          // leader's arrivals as well: a fixed time for them to land
          const uint64_t t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 200000ull) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (one thread of the leader)
    if (lane == 0 && leader) {
      uint32_t stage = 0, phase = 0, local = 0;
      bool ok = true;
      // K-major: 8-row groups 1024 bytes apart, 32 bytes a step of K.  MN-major: 64
      // channels x 8 K rows are 1024 bytes, the next 64 channels 8192 on, 16 K rows a step.
      const uint64_t a_desc = umma_desc_sw128(smem_u32(smem), A_MN ? 8192 : 16, 1024);
      const uint64_t b_desc = umma_desc_sw128(smem_u32(smem) + C::OPERAND, B_MN ? 8192 : 16, 1024);
      for (int item = first; ok && item < P.items; item += stride, ++local) {
        const uint32_t acc = local & 1, aphase = (local >> 1) & 1;
        ok = mbar_wait(&tempty[acc], aphase ^ 1, abort_flag, err, 12);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * C::BN;
        // The issuer does without the tile's place where it can: with the divisions of
        // tile_of and of a split's bounds the tensor cores waited longer
        // between tiles: the video case took 978 us instead of 960, from e4m3 577 instead of 550.
        int kb0 = 0, kb1 = P.k_blocks;
        if (P.splits > 1) {
          kb0 = item / (P.m_tiles * P.n_tiles) % P.splits * P.k_per;
          kb1 = min(kb1, kb0 + P.k_per);
        }
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = mbar_wait(&full[stage], phase, abort_flag, err, 13);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = umma_desc_add(a_desc, stage * C::STAGE), bd = umma_desc_add(b_desc, stage * C::STAGE);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t ak = umma_desc_add(ad, k * (A_MN ? 2048 : 32)), bk = umma_desc_add(bd, k * (B_MN ? 2048 : 32));
            const uint32_t accum = kb > kb0 || k > 0;
            if constexpr (PAIR && F8) umma_ss_f8_pair(d, ak, bk, P.idesc, accum);
            else if constexpr (PAIR) umma_ss_pair(d, ak, bk, P.idesc, accum);
            else if constexpr (F8) umma_ss_f8(d, ak, bk, P.idesc, accum);
            else umma_ss(d, ak, bk, P.idesc, accum);
          }
          if constexpr (PAIR) umma_commit_pair(&empty[stage], 0x3);
          else umma_commit(&empty[stage]);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if constexpr (PAIR) umma_commit_pair(&tfull[acc], 0x3);
        else umma_commit(&tfull[acc]);
      }
      if (!ok) abort_pair();
      // every MMA of this thread completes before tensor memory is freed
      if constexpr (PAIR) umma_commit_pair(drained, 0x1);
      else umma_commit(drained);
      volatile int no_abort = 0;
      mbar_wait(drained, 0, &no_abort, nullptr, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ draining warps
    const int q = warp & 3, half = (warp - 2) / 4;
    uint8_t* stg = smem + C::STG_OFF + (warp - 2) * C::STG;
    const uint32_t tempty_leader = PAIR ? cluster_map(tempty, 0) : 0;
    uint32_t local = 0;
    bool ok = true;
    for (int item = first; item < P.items; item += stride, ++local) {
      const uint32_t acc = local & 1, aphase = (local >> 1) & 1;
      ok = mbar_wait_warp(&tfull[acc], aphase, abort_flag, err, 14);
      if (!ok) break;
      tc_fence_after();
      const Tile t = tile_of(P, item);
      const int64_t row0 = (PAIR ? (int64_t)(2 * t.mb + (int)rank) * C::BM : (int64_t)t.mb * C::BM) + q * 32;
      auto release = [&]() {
        if constexpr (PAIR) mbar_arrive_cluster(tempty_leader + acc * (uint32_t)sizeof(uint64_t));
        else mbar_arrive(&tempty[acc]);
      };
      drain<MODE, F8, ACT, C::BN>(P, t, tmem_base + acc * C::BN + ((uint32_t)(q * 32) << 16), row0, half, stg, release);
    }
    if (!ok && lane == 0) abort_pair();
    if (lane == 0) bulk_wait0();  // this warp's tensor stores have landed
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // a pair frees its tensor memory together, when neither CTA has remote arrivals
  // or copies left to make into the other
  if constexpr (PAIR) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- few rows
// Forward of at most 32 rows: both weights are all there is to read.  A block takes
// 16 hidden channels, its warps a part of K each, and every lane fetches 16-byte
// pieces of the weights' rows straight into registers, four steps at a time.  The
// products run on mma.m16n8k16 with the channels as rows and 8 tokens as columns: a
// lane's eight neighbours in K serve as the fragment's scattered ones, of x alike.
// e4m3 is widened to fp16, which holds it exactly.
struct Few {
  const uint8_t *x, *w[2];
  int64_t ldx, ldw[2];  // bytes
  const float *x_scale, *scale[2], *bias[2];
  uint16_t* out[3];
  int64_t ldo[3];       // elements
  int M, D, F;
};
constexpr int kFewWarps = 4, kFewRows = 32;

// 16 bytes of a row from element k on (k a multiple of 16 bytes), zeros from D on.
// WHOLE: D and the row's address are multiples of 16 bytes.
template <bool F8, bool WHOLE>
DIT_DEV uint4 piece(const uint8_t* row, int k, int D) {
  constexpr int E = F8 ? 16 : 8;
  if (WHOLE) {
    if (k < D) return __ldg(reinterpret_cast<const uint4*>(row + k * (16 / E)));
    return make_uint4(0, 0, 0, 0);
  }
  if constexpr (F8) return k < D ? load16(row, k, D) : make_uint4(0, 0, 0, 0);
  // eight loads of 2 bytes: 92 us for 20 rows x 4095 x 8191, 104 by shifted vectors
  // (of e4m3, sixteen loads of a byte: 97 us, by shifted vectors 61)
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < E; ++j)
    if (k + j < D) w[(j / 2) & 3] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(row) + k + j) << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
DIT_DEV uint32_t widen(uint32_t two_e4m3) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two_e4m3));
  return h;
}
template <bool F16>
DIT_DEV void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c += the 16 channels' pieces (rows g and g + 8) x 8 tokens' pieces
template <bool F8, bool F16>
DIT_DEV void products(float (&c)[4], const uint4& lo, const uint4& hi, const uint4& x) {
  const uint32_t *a = &lo.x, *b = &hi.x, *t = &x.x;
  if constexpr (F8) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      mma16816<true>(c, widen(a[j]), widen(b[j]), widen(a[j] >> 16), widen(b[j] >> 16), widen(t[j]), widen(t[j] >> 16));
  } else {
#pragma unroll
    for (int j = 0; j < 4; j += 2) mma16816<F16>(c, a[j], b[j], a[j + 1], b[j + 1], t[j], t[j + 1]);
  }
}

// NT: groups of 8 tokens.  F16: the output's type, and of 16-bit operands theirs.
// BLOCKS: an SM's; with five of them, fewer pieces are under way in each.
template <bool F8, bool F16, int NT, bool WHOLE, int ACT, int BLOCKS>
__global__ void __launch_bounds__(32 * kFewWarps, BLOCKS) few_rows_kernel(const Few a) {
  constexpr int E = F8 ? 16 : 8, STEP = 4 * E, U = NT > 2 || (F8 && !WHOLE) || BLOCKS > 4 ? 2 : 4;
  __shared__ float sums[2][kFewWarps][NT][16][9];
  wait_previous();
  start_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int f0 = blockIdx.x * 16;
  const int steps = (a.D + STEP - 1) / STEP;
  const int s0 = steps * warp / kFewWarps, s1 = steps * (warp + 1) / kFewWarps;
  const uint8_t* rows[2][2];  // of channels that are not there: the last one's (never stored)
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    rows[m][0] = a.w[m] + min(f0 + g, a.F - 1) * a.ldw[m];
    rows[m][1] = a.w[m] + min(f0 + g + 8, a.F - 1) * a.ldw[m];
  }
  float acc[2][NT][4] = {};
  for (int s = s0; s < s1; s += U) {
    uint4 w[U][2][2], x[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = s + u < s1 ? (s + u) * STEP + t * E : a.D;  // from D on: zeros
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        w[u][m][0] = piece<F8, WHOLE>(rows[m][0], k, a.D);
        w[u][m][1] = piece<F8, WHOLE>(rows[m][1], k, a.D);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) x[u][n] = piece<F8, WHOLE>(a.x + (n * 8 + g) * a.ldx, n * 8 + g < a.M ? k : a.D, a.D);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) products<F8, F16>(acc[m][n], w[u][m][0], w[u][m][1], x[u][n]);
  }
  // accumulator element (row g or g + 8, token 2 t or 2 t + 1)
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) sums[m][warp][n][g + (j >> 1) * 8][2 * t + (j & 1)] = acc[m][n][j];
  __syncthreads();
  for (int i = threadIdx.x; i < 128 * NT; i += 32 * kFewWarps) {
    const int c = i & 15, tok = (i >> 4) & 7, n = i >> 7;
    const int row = n * 8 + tok, f = f0 + c;
    if (row >= a.M || f >= a.F) continue;
    float v[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      v[m] = sums[m][0][n][c][tok];
#pragma unroll
      for (int w = 1; w < kFewWarps; ++w) v[m] += sums[m][w][n][c][tok];
      if constexpr (F8) v[m] = v[m] * __ldg(a.scale[m] + f) * __ldg(a.x_scale + row);
      if (a.bias[m]) v[m] += __ldg(a.bias[m] + f);
      if (a.out[1]) a.out[1 + m][row * a.ldo[1 + m] + f] = (uint16_t)pack16(F16, v[m], 0.f);
    }
    const float2 h = gated2<ACT>(make_float2(v[0], v[0]), make_float2(v[1], v[1]));
    a.out[0][row * a.ldo[0] + f] = (uint16_t)pack16(F16, h.x, 0.f);
  }
}

// ---------------------------------------------------------------- partial sums
struct Join {
  const float* partial;  // planes [problem][split][side]
  int64_t ldp, plane;
  int splits;
  const float *x_scale, *scale[2], *bias[2];
  void* out[3];
  int64_t ldo[3];
  int64_t M;
  int N;
  int f16, act;
  int late;  // the kernels before the previous one have written what is read (launch.cuh)
};

DIT_DEV void store4(void* base, int64_t at, int n, int f16, const float (&v)[4]) {
  uint16_t* p = static_cast<uint16_t*>(base) + at;
  const uint32_t a = pack16(f16, v[0], v[1]), b = pack16(f16, v[2], v[3]);
  if (n >= 4 && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
    *reinterpret_cast<uint2*>(p) = make_uint2(a, b);
    return;
  }
  p[0] = (uint16_t)a;
  if (n > 1) p[1] = (uint16_t)(a >> 16);
  if (n > 2) p[2] = (uint16_t)b;
  if (n > 3) p[3] = (uint16_t)(b >> 16);
}
DIT_DEV void sum_planes(const float* p, int64_t step, int n, float (&v)[4]) {
  float4 s = __ldcg(reinterpret_cast<const float4*>(p));
#pragma unroll 4
  for (int z = 1; z < n; ++z) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(p + z * step));
    s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
  }
  v[0] = s.x, v[1] = s.y, v[2] = s.z, v[3] = s.w;
}
// The splits of K joined in order, four columns a thread, then what the tile's
// epilogue would have done.  blockIdx.z: the problem.
template <bool GATED>
__global__ void __launch_bounds__(256) join_kernel(const Join J) {
  if (!J.late) wait_previous();
  start_next();
  const int64_t groups = J.ldp / 4, total = J.M * groups;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t row = i / groups;
    const int c = (int)(i - row * groups) * 4;
    const int n = J.N - c;
    const float* p = J.partial + row * J.ldp + c;
    float v[4];
    if constexpr (GATED) {
      float g[4];
      sum_planes(p, 2 * J.plane, J.splits, g);
      sum_planes(p + J.plane, 2 * J.plane, J.splits, v);
      const float rs = J.x_scale ? __ldg(J.x_scale + row) : 1.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= n) continue;
        if (J.scale[0]) g[j] = g[j] * __ldg(J.scale[0] + c + j) * rs, v[j] = v[j] * __ldg(J.scale[1] + c + j) * rs;
        if (J.bias[0]) g[j] += __ldg(J.bias[0] + c + j);
        if (J.bias[1]) v[j] += __ldg(J.bias[1] + c + j);
      }
      if (J.out[1]) {
        store4(J.out[1], row * J.ldo[1] + c, n, J.f16, g);
        store4(J.out[2], row * J.ldo[2] + c, n, J.f16, v);
      }
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float2 a = make_float2(g[j], g[j + 1]), b = make_float2(v[j], v[j + 1]);
        const float2 h = J.act == DIT_ACT_SILU ? gated2<DIT_ACT_SILU>(a, b) : gated2<DIT_ACT_GELU>(a, b);
        v[j] = h.x, v[j + 1] = h.y;
      }
      store4(J.out[0], row * J.ldo[0] + c, n, J.f16, v);
    } else {
      sum_planes(p + (int64_t)blockIdx.z * J.splits * J.plane, J.plane, J.splits, v);
      store4(J.out[blockIdx.z], row * J.ldo[blockIdx.z] + c, n, J.f16, v);
    }
  }
  if (J.late) wait_previous();
}

// ---------------------------------------------------------------- copies of unaligned operands
struct Pack {
  const uint8_t* src[3];
  uint8_t* dst[3];
  int64_t rows[3], src_stride[3];
  int width;  // elements
  int64_t pitch;
};
// Rows of any alignment to rows at multiples of 16 bytes (blockIdx.y: operand).
template <typename E>
__global__ void __launch_bounds__(256) pack_kernel(const Pack a) {
  wait_previous();
  start_next();
  const int o = blockIdx.y;
  if (!a.src[o]) return;
  const E* src = reinterpret_cast<const E*>(a.src[o]);
  E* dst = reinterpret_cast<E*>(a.dst[o]);
  // a warp per row, a vector a lane; the pitch is one of whole vectors
  constexpr int PER = 16 / sizeof(E);
  const int lane = threadIdx.x & 31;
  for (int64_t r = (blockIdx.x * 256ll + threadIdx.x) >> 5; r < a.rows[o]; r += gridDim.x * 8ll)
#pragma unroll 4
    for (int c = lane * PER; c < a.width; c += 32 * PER)
      *reinterpret_cast<uint4*>(dst + r * a.pitch + c) = load16(src + r * a.src_stride[o], c, a.width);
}

// ---------------------------------------------------------------- gradients of gate and up
struct Slopes {
  const uint16_t *gate, *up, *dout;
  int64_t ld_gate, ld_up, ld_dout;
  uint16_t *dgate, *dup;  // at multiples of 16 bytes
  int64_t pitch;
  float* partial;         // [row block][2][pitch] sums of the block's rows, or NULL
  int64_t M;
  int F, rows_per_block;
};

// Eight values at p, of which n are there (zeros behind them).  ALIGN: bytes that rows
// and addresses are multiples of; at 16 and 4 the number of values is a multiple too.
// (Shifted vectors at the alignment of 2 took the odd case's slopes 14 us, these 8.)
template <int ALIGN>
DIT_DEV uint4 load8(const uint16_t* p, int n) {
  if constexpr (ALIGN == 16) {
    return __ldcs(reinterpret_cast<const uint4*>(p));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (ALIGN == 4) w[j] = 2 * j < n ? __ldcs(reinterpret_cast<const uint32_t*>(p) + j) : 0u;
      else w[j] = (2 * j < n ? (uint32_t)p[2 * j] : 0u) | (2 * j + 1 < n ? (uint32_t)p[2 * j + 1] << 16 : 0u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// 256 columns (8 a lane) x rows_per_block rows a block, 8 x ROWS rows at a time.  dgate and
// dup are rounded to the type: the tensor cores want both operands of a product in it, and
// x and the weights are there.  That leaves dx and the weights' gradients 2.35e-3 of their
// norm off in bf16 and 2.9e-4 in fp16, where their own rounding alone makes 1.66e-3 and
// 2.1e-4; tf32 operands would keep all but run at half the rate on twice the bytes, of
// widened copies of x and the weights too.  The bias sums take them unrounded.
template <typename T, int ACT, int ALIGN>
__global__ void __launch_bounds__(256) slopes_kernel(const Slopes a) {
  constexpr int ROWS = 2;
  __shared__ float sums[8][2][32][9];
  wait_previous();
  start_next();
  const int lane = threadIdx.x, ty = threadIdx.y;
  const int c = (blockIdx.y * 32 + lane) * 8;
  const int n = a.F - c;
  float sg[8] = {}, su[8] = {};
  const int64_t r0 = (int64_t)blockIdx.x * a.rows_per_block;
  const int64_t r1 = min(a.M, r0 + a.rows_per_block);
  if (n > 0) {
    for (int64_t r = r0 + ty; r < r1; r += 8 * ROWS) {
      uint4 raw[ROWS][3];
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        const int64_t at = r + 8 * k;
        if (at >= r1) continue;
        raw[k][0] = load8<ALIGN>(a.gate + at * a.ld_gate + c, n);
        raw[k][1] = load8<ALIGN>(a.up + at * a.ld_up + c, n);
        raw[k][2] = load8<ALIGN>(a.dout + at * a.ld_dout + c, n);
      }
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        const int64_t at = r + 8 * k;
        if (at >= r1) continue;
        const uint32_t *pg = &raw[k][0].x, *pu = &raw[k][1].x, *pd = &raw[k][2].x;
        uint32_t wg[4], wu[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 g = unpack2<T>(pg[j]), u = unpack2<T>(pu[j]), d = unpack2<T>(pd[j]);
          const float2 s0 = activation_slope<ACT>(g.x), s1 = activation_slope<ACT>(g.y);
          float2 dg = fmul2(fmul2(d, u), make_float2(s0.y, s1.y)), du = fmul2(d, make_float2(s0.x, s1.x));
          if (ALIGN < 16 && 2 * j >= n) dg.x = du.x = 0.f;
          if (ALIGN < 16 && 2 * j + 1 >= n) dg.y = du.y = 0.f;
          sg[2 * j] += dg.x, sg[2 * j + 1] += dg.y;
          su[2 * j] += du.x, su[2 * j + 1] += du.y;
          wg[j] = pack2<T>(dg.x, dg.y);
          wu[j] = pack2<T>(du.x, du.y);
        }
        // c + 8 <= pitch: the pitch is a multiple of 8
        *reinterpret_cast<uint4*>(a.dgate + at * a.pitch + c) = make_uint4(wg[0], wg[1], wg[2], wg[3]);
        *reinterpret_cast<uint4*>(a.dup + at * a.pitch + c) = make_uint4(wu[0], wu[1], wu[2], wu[3]);
      }
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[ty][0][lane][j] = sg[j], sums[ty][1][lane][j] = su[j];
  __syncthreads();
  // 512 sums (2 sides x 256 columns), two a thread
  for (int i = ty * 32 + lane; i < 512; i += 256) {
    const int side = i >> 8, col = i & 255;
    float v = 0.f;
#pragma unroll
    for (int y = 0; y < 8; ++y) v += sums[y][side][col >> 3][col & 7];
    const int64_t at = blockIdx.y * 256 + col;
    if (at < a.pitch / 2) a.partial[((int64_t)blockIdx.x * 2 + side) * (a.pitch / 2) + at] = v;
  }
}

// ---------------------------------------------------------------- plan
int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// How a product runs: tiles and splits of K.
struct Split {
  bool pair;
  int splits;
};
// The fewest estimated cycles over both tile shapes and 1 .. 16 splits.  A K block
// costs a pair 512 cycles on 256 x 256 (the tensor cores' rate), a single CTA
// about 300 on 128 x 128 (256 at that rate); a launch fills and drains in about 4000,
// and partial sums cost their traffic (written and read, fp32) and a launch.
//
// No split is longer than kLongest blocks, 4096 steps of the tensor cores (65536 terms of 16
// bits, 131072 of e4m3): their fp32 sums lose up to 2^-23 of themselves at each step, to
// one side (16.8 M rows of terms of one sign, 1 M a split: dW 6.6e-3 too small), and a
// wait for a tile has a limit in time.
constexpr int64_t kLongest = 1024;
Split choose(int64_t M, int64_t N, int64_t cols_per_n, int64_t k_blocks, int problems) {
  Split best{false, 1};
  double least = 0;
  const int64_t fewest = (k_blocks + kLongest - 1) / kLongest;
  for (int pair = 0; pair < 2; ++pair)
    for (int64_t s = fewest > 1 ? fewest : 1; s <= fewest || s <= 16; ++s) {
      if (s > 1 && s > fewest && k_blocks / s < 4) break;
      const int64_t per = (k_blocks + s - 1) / s;
      const int64_t splits = (k_blocks + per - 1) / per;  // none is empty
      const int64_t tm = pair ? 256 : 128, tn = (pair ? 256 : 128) / cols_per_n;
      const int64_t tiles = ((M + tm - 1) / tm) * ((N + tn - 1) / tn) * problems * splits;
      const int64_t slots = pair ? kSms / 2 : kSms;
      double t = (double)((tiles + slots - 1) / slots) * (double)per * (pair ? 512. : 300.) + 4000.;
      if (splits > 1) t += 5000. + (double)M * N * cols_per_n * problems * splits * 8. / 3500.;
      if (least == 0 || t < least) least = t, best = Split{pair != 0, (int)splits};
    }
  return best;
}

constexpr int64_t kMaxStride = (int64_t)1 << 40;  // bytes
struct Operand {
  const void* p;
  int64_t stride;
  bool packed;    // copied to `offset` of the workspace, rows of `pitch` elements
  int64_t offset, pitch;
};
struct Plan {
  Operand x, wg, wu;
  Split fwd, dx, dw;
  bool few = false;
  int64_t slopes = -1, slope_pitch = 0;   // [rows][2][pitch] 16-bit
  int64_t sums = -1, sum_blocks = 0, rows_per_block = 0;
  int64_t partial = -1, partial_dw = -1;
  int64_t bytes = 0;
  int64_t take(int64_t n) {
    const int64_t at = bytes;
    bytes += round_up(n, 256);
    return at;
  }
};
int64_t planes(const Split& s, int64_t M, int64_t N, int sides) {
  return s.splits > 1 ? (int64_t)s.splits * sides * M * round_up(N, 4) * 4 : 0;
}
Plan make_plan(const dit_gated_ffn_args& a, bool backward) {
  Plan p;
  const int esz = a.operand_dtype == DIT_DTYPE_E4M3 ? 1 : 2;
  p.few = !backward && a.rows <= kFewRows;
  auto operand = [&](Operand& o, const void* ptr, int64_t stride, int64_t rows, bool used) {
    o.p = ptr, o.stride = stride;
    if (rows <= 1) o.stride = round_up(a.width, 16 / esz);  // the stride of a single row says nothing
    // as a tensor map wants them: 16-byte rows, strides below 2^40 bytes; rows that overlap are no matrix
    o.packed = used && !p.few && ((((uintptr_t)ptr | (uintptr_t)(o.stride * esz)) & 15) != 0 || o.stride < a.width ||
                        o.stride * esz >= kMaxStride);
    o.pitch = round_up(a.width, 16 / esz);
    o.offset = o.packed ? p.take(rows * o.pitch * esz) : 0;
  };
  operand(p.x, a.x, a.x_stride, a.rows, !backward || a.dw_gate || a.dw_up);
  operand(p.wg, a.w_gate, a.w_gate_stride, a.hidden, !backward || a.dx);
  operand(p.wu, a.w_up, a.w_up_stride, a.hidden, !backward || a.dx);
  const int bk = 128 / esz;
  if (p.few) return p;
  if (!backward) {
    p.fwd = choose(a.rows, a.hidden, 2, (a.width + bk - 1) / bk, 1);
    if (p.fwd.splits > 1) p.partial = p.take(planes(p.fwd, a.rows, a.hidden, 2));
    return p;
  }
  p.slope_pitch = round_up(a.hidden, 8);
  p.slopes = p.take(a.rows * p.slope_pitch * 2 * 2);
  // few rows a block while there are few blocks; at most 32 serial additions either way
  p.rows_per_block = a.rows * a.hidden > (1 << 24) ? 256 : a.rows * a.hidden > (1 << 21) ? 32 : 16;
  p.sum_blocks = (a.rows + p.rows_per_block - 1) / p.rows_per_block;
  if (a.dbias_gate || a.dbias_up) p.sums = p.take(p.sum_blocks * 2 * p.slope_pitch * 4);
  const int problems = (a.dw_gate ? 1 : 0) + (a.dw_up ? 1 : 0);
  if (a.dx) {
    p.dx = choose(a.rows, a.width, 1, 2 * ((a.hidden + 63) / 64), 1);
    if (p.dx.splits > 1) p.partial = p.take(planes(p.dx, a.rows, a.width, 1));
  }
  if (problems) {
    p.dw = choose(a.hidden, a.width, 1, (a.rows + 63) / 64, problems);
    if (p.dw.splits > 1) p.partial_dw = p.take(planes(p.dw, a.hidden, a.width, problems));
  }
  return p;
}

// ---------------------------------------------------------------- launches
// CTAs, or pairs of them, that run at once on the current device: a persistent
// launch asks for no more (one that had to wait would run its whole share last).
template <int MODE, bool F8, bool PAIR, int ACT>
cudaError_t resident(int* slots) {
  static int known[kMaxDevices] = {};  // 0: not asked yet; every thread finds the same number
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int n = __atomic_load_n(&known[dev], __ATOMIC_RELAXED);
  if (n == 0) {
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    n = sms;
    if (PAIR) {
      using C = Cfg<F8, PAIR>;
      const auto kernel = product_kernel<MODE, F8, PAIR, ACT>;
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 << 10);
      if (e != cudaSuccess) return e;
      cudaLaunchConfig_t c{};
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = 2;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      c.gridDim = dim3(2 * (sms / 2));
      c.blockDim = dim3(kThreads);
      c.dynamicSmemBytes = C::SMEM;
      c.attrs = at;
      c.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&n, kernel, &c);
      if (e != cudaSuccess) return e;
      if (n > sms / 2) n = sms / 2;
    }
    if (n < 1) return cudaErrorLaunchOutOfResources;
    __atomic_store_n(&known[dev], n, __ATOMIC_RELAXED);
  }
  *slots = n;
  return cudaSuccess;
}

template <int MODE, bool F8, bool PAIR, int ACT>
cudaError_t launch_product(Product& P, int problems, cudaStream_t s) {
  using C = Cfg<F8, PAIR>;
  constexpr int COLS = MODE == FWD ? C::BN / 2 : C::BN;
  P.m_tiles = (int)((P.M + C::TILE_M - 1) / C::TILE_M);
  P.n_tiles = (P.N + COLS - 1) / COLS;
  P.items = P.m_tiles * P.n_tiles * P.splits * problems;
  const int mma_m = C::MMA_M;
  P.idesc = F8 ? umma_idesc_e4m3(mma_m, C::BN) : umma_idesc_bf16(mma_m, C::BN, MODE != FWD);
  if (MODE == DW) P.idesc |= 1u << 15;              // A lies across K too
  if (!F8 && P.f16) P.idesc &= ~((1u << 7) | (1u << 10));  // format 0: f16
  // column groups whose part of B is at most 40 MB, while A is no larger than B
  const int64_t k_bytes = (int64_t)P.k_blocks * 128;
  int64_t gn = ((int64_t)40 << 20) / (k_bytes * C::BN);
  if (gn < 1) gn = 1;
  if (P.M * 1 > (int64_t)P.N * (MODE == FWD ? 2 : 1) || gn > P.n_tiles) gn = P.n_tiles;
  P.group_n = (int)gn;
  int slots = 0;
  const cudaError_t e = resident<MODE, F8, PAIR, ACT>(&slots);
  if (e != cudaSuccess) return e;
  const int n = P.items < slots ? P.items : slots;
  return launch_kernel(product_kernel<MODE, F8, PAIR, ACT>, dim3(PAIR ? 2 * n : n), dim3(kThreads), C::SMEM, s, PAIR ? 2 : 1, true, P);
}
template <int MODE, bool F8>
cudaError_t run_product(Product& P, const Split& sp, int problems, cudaStream_t s) {
  P.splits = sp.splits;
  P.k_per = (P.k_blocks + sp.splits - 1) / sp.splits;
  if constexpr (MODE == FWD)
    if (P.act == DIT_ACT_GELU)
      return sp.pair ? launch_product<MODE, F8, true, DIT_ACT_GELU>(P, problems, s) : launch_product<MODE, F8, false, DIT_ACT_GELU>(P, problems, s);
  return sp.pair ? launch_product<MODE, F8, true, DIT_ACT_SILU>(P, problems, s) : launch_product<MODE, F8, false, DIT_ACT_SILU>(P, problems, s);
}

// rows x width elements: boxes of 128 bytes (box_x elements) by box_rows rows
bool operand_map(CUtensorMap* m, int f8, int f16, const void* p, int64_t width, int64_t rows, int64_t stride, int box_rows) {
  const int esz = f8 ? 1 : 2;
  const uint64_t d[2] = {(uint64_t)width, (uint64_t)rows}, st[1] = {(uint64_t)stride * esz};
  const uint32_t box[2] = {(uint32_t)(128 / esz), (uint32_t)box_rows};
  const CUtensorMapDataType t = f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return make_tmap(m, t, p, 2, d, st, box);
}
// An output: by tensor stores where its alignment lets them.
void output(Product& P, int o, void* p, int64_t ld) {
  P.out[o] = p, P.ldo[o] = ld;
  P.tma[o] = 0;
  if (!p || (uintptr_t)p % 16 || (P.M > 1 && (ld % 8 || ld * 2 >= kMaxStride)) || P.splits > 1) return;
  const int64_t stride = P.M > 1 ? ld : round_up(P.N, 8);
  P.tma[o] = operand_map(&P.c[o], 0, P.f16, p, P.N, P.M, stride, 32);
}

template <bool GATED>
cudaError_t join(const Product& P, int problems, bool late, cudaStream_t s) {
  Join J{P.partial, P.ldp, P.plane, P.splits, P.x_scale, {P.scale[0], P.scale[1]}, {P.bias[0], P.bias[1]},
         {P.out[0], P.out[1], P.out[2]}, {P.ldo[0], P.ldo[1], P.ldo[2]}, P.M, P.N, P.f16, P.act, late};
  const int64_t blocks = (P.M * (P.ldp / 4) + 255) / 256;
  return launch_kernel(join_kernel<GATED>, dim3((unsigned)(blocks < kSms * 16 ? blocks : kSms * 16), 1, problems), dim3(256), 0, s, 1, true, J);
}

cudaError_t pack_operands(const dit_gated_ffn_args& a, Plan& p, char* ws, cudaStream_t s) {
  Pack k{};
  const int esz = a.operand_dtype == DIT_DTYPE_E4M3 ? 1 : 2;
  Operand* ops[3] = {&p.x, &p.wg, &p.wu};
  const int64_t rows[3] = {a.rows, a.hidden, a.hidden};
  bool any = false;
  k.width = a.width;
  int64_t most = 0;
  for (int i = 0; i < 3; ++i) {
    Operand& o = *ops[i];
    if (!o.packed) continue;
    any = true;
    k.src[i] = static_cast<const uint8_t*>(o.p);
    k.dst[i] = reinterpret_cast<uint8_t*>(ws + o.offset);
    k.rows[i] = rows[i], k.src_stride[i] = o.stride, k.pitch = o.pitch;
    most = rows[i] > most ? rows[i] : most;
    o.p = k.dst[i], o.stride = o.pitch;
  }
  if (!any) return cudaSuccess;
  const dim3 grid((unsigned)((most + 7) / 8 < kSms * 8 ? (most + 7) / 8 : kSms * 8), 3);
  return esz == 1 ? launch_kernel(pack_kernel<uint8_t>, grid, dim3(256), 0, s, 1, false, k)
                  : launch_kernel(pack_kernel<uint16_t>, grid, dim3(256), 0, s, 1, false, k);
}

// Five blocks an SM where four of each would be more than one round: 11008 channels
// from width 4096 for 1 / 16 / 32 rows 31 / 32 / 37 us instead of 32 / 40 / 49; where
// four are enough they are as good or better (8960 from 1536: 32 rows 13 us, 16 with five).
template <bool F8, bool F16, int NT, int ACT>
cudaError_t launch_few(const Few& k, bool whole, cudaStream_t s) {
  const int blocks = (k.F + 15) / 16;
  const auto kernel = !whole                ? few_rows_kernel<F8, F16, NT, false, ACT, 4>
                      : blocks > 4 * kSms   ? few_rows_kernel<F8, F16, NT, true, ACT, 5>
                                            : few_rows_kernel<F8, F16, NT, true, ACT, 4>;
  return launch_kernel(kernel, dim3(blocks), dim3(32 * kFewWarps), 0, s, 1, true, k);
}
template <bool F8, bool F16, int NT>
cudaError_t launch_few(const Few& k, bool whole, int act, cudaStream_t s) {
  return act == DIT_ACT_SILU ? launch_few<F8, F16, NT, DIT_ACT_SILU>(k, whole, s) : launch_few<F8, F16, NT, DIT_ACT_GELU>(k, whole, s);
}
template <bool F8, bool F16>
cudaError_t launch_few(const Few& k, bool whole, int act, cudaStream_t s) {
  if (k.M <= 8) return launch_few<F8, F16, 1>(k, whole, act, s);
  if (k.M <= 16) return launch_few<F8, F16, 2>(k, whole, act, s);
  return launch_few<F8, F16, 4>(k, whole, act, s);
}
cudaError_t few_rows(const dit_gated_ffn_args& a, cudaStream_t s) {
  const bool f8 = a.operand_dtype == DIT_DTYPE_E4M3, f16 = a.dtype == DIT_DTYPE_F16;
  const int esz = f8 ? 1 : 2;
  Few k{};
  k.x = static_cast<const uint8_t*>(a.x), k.w[0] = static_cast<const uint8_t*>(a.w_gate), k.w[1] = static_cast<const uint8_t*>(a.w_up);
  k.ldx = a.rows > 1 ? a.x_stride * esz : 0;
  k.ldw[0] = a.hidden > 1 ? a.w_gate_stride * esz : 0, k.ldw[1] = a.hidden > 1 ? a.w_up_stride * esz : 0;
  k.x_scale = a.x_scale, k.scale[0] = a.gate_scale, k.scale[1] = a.up_scale;
  k.bias[0] = a.bias_gate, k.bias[1] = a.bias_up;
  k.out[0] = static_cast<uint16_t*>(a.out), k.out[1] = static_cast<uint16_t*>(a.gate), k.out[2] = static_cast<uint16_t*>(a.up);
  k.ldo[0] = a.out_stride, k.ldo[1] = a.gate_stride, k.ldo[2] = a.up_stride;
  k.M = (int)a.rows, k.D = a.width, k.F = a.hidden;
  const uint64_t all = (uintptr_t)k.x | (uintptr_t)k.w[0] | (uintptr_t)k.w[1] | (uint64_t)(k.ldx | k.ldw[0] | k.ldw[1]) | (uint64_t)(a.width * esz);
  const bool whole = (all & 15) == 0;
  if (f8) return f16 ? launch_few<true, true>(k, whole, a.act, s) : launch_few<true, false>(k, whole, a.act, s);
  return f16 ? launch_few<false, true>(k, whole, a.act, s) : launch_few<false, false>(k, whole, a.act, s);
}

cudaError_t forward(const dit_gated_ffn_args& a, char* ws, cudaStream_t s) {
  Plan p = make_plan(a, false);
  if (p.few) return few_rows(a, s);
  cudaError_t e = pack_operands(a, p, ws, s);
  if (e != cudaSuccess) return e;
  const bool f8 = a.operand_dtype == DIT_DTYPE_E4M3;
  Product P{};
  P.M = a.rows, P.N = a.hidden;
  P.f16 = a.dtype == DIT_DTYPE_F16, P.act = a.act;
  P.k_blocks = (a.width + (f8 ? 127 : 63)) / (f8 ? 128 : 64);
  P.k_half = P.k_blocks;
  P.splits = p.fwd.splits;
  P.x_scale = a.x_scale, P.scale[0] = a.gate_scale, P.scale[1] = a.up_scale;
  P.bias[0] = a.bias_gate, P.bias[1] = a.bias_up;
  if (p.fwd.splits > 1) P.partial = reinterpret_cast<float*>(ws + p.partial);
  P.ldp = round_up(P.N, 4), P.plane = P.M * P.ldp;
  const int brows = p.fwd.pair ? 128 : 64;
  if (!operand_map(&P.a[0], f8, P.f16, p.x.p, a.width, a.rows, p.x.stride, 128) ||
      !operand_map(&P.b[0], f8, P.f16, p.wg.p, a.width, a.hidden, p.wg.stride, brows) ||
      !operand_map(&P.b[1], f8, P.f16, p.wu.p, a.width, a.hidden, p.wu.stride, brows))
    return cudaErrorInvalidValue;
  output(P, 0, a.out, a.out_stride);
  output(P, 1, a.gate, a.gate_stride);
  output(P, 2, a.up, a.up_stride);
  e = f8 ? run_product<FWD, true>(P, p.fwd, 1, s) : run_product<FWD, false>(P, p.fwd, 1, s);
  return e != cudaSuccess || P.splits == 1 ? e : join<true>(P, 1, false, s);
}

template <typename T>
cudaError_t run_slopes(const Slopes& g, int act, cudaStream_t s) {
  const uintptr_t all = (uintptr_t)g.gate | (uintptr_t)g.up | (uintptr_t)g.dout;
  const int64_t steps = g.M > 1 ? g.ld_gate | g.ld_up | g.ld_dout : 0;
  const uint64_t at = all | (uint64_t)(steps * 2) | (uint64_t)g.F * 2;
  const dim3 grid((unsigned)((g.M + g.rows_per_block - 1) / g.rows_per_block), (unsigned)((g.F + 255) / 256));
  const auto kernel = act == DIT_ACT_SILU ? at % 16 == 0  ? slopes_kernel<T, DIT_ACT_SILU, 16>
                                            : at % 4 == 0 ? slopes_kernel<T, DIT_ACT_SILU, 4> : slopes_kernel<T, DIT_ACT_SILU, 2>
                      : at % 16 == 0 ? slopes_kernel<T, DIT_ACT_GELU, 16>
                      : at % 4 == 0  ? slopes_kernel<T, DIT_ACT_GELU, 4> : slopes_kernel<T, DIT_ACT_GELU, 2>;
  return launch_kernel(kernel, grid, dim3(32, 8), 0, s, 1, true, g);
}

cudaError_t zero_rows(void* p, int64_t rows, int64_t width, int64_t stride, cudaStream_t s) {
  if (!p) return cudaSuccess;
  return cudaMemset2DAsync(p, (size_t)(rows > 1 ? stride : width) * 2, 0, (size_t)width * 2, (size_t)rows, s);
}

cudaError_t backward(const dit_gated_ffn_args& a, char* ws, cudaStream_t s) {
  if (a.rows == 0) {
    cudaError_t e = zero_rows(a.dw_gate, a.hidden, a.width, a.dw_gate_stride, s);
    if (e == cudaSuccess) e = zero_rows(a.dw_up, a.hidden, a.width, a.dw_up_stride, s);
    for (float* b : {a.dbias_gate, a.dbias_up})
      if (e == cudaSuccess && b) e = cudaMemsetAsync(b, 0, (size_t)a.hidden * 4, s);
    return e;
  }
  Plan p = make_plan(a, true);
  cudaError_t e = pack_operands(a, p, ws, s);
  if (e != cudaSuccess) return e;
  const int f16 = a.dtype == DIT_DTYPE_F16;
  Slopes g{};
  g.gate = static_cast<const uint16_t*>(a.gate), g.up = static_cast<const uint16_t*>(a.up);
  g.dout = static_cast<const uint16_t*>(a.out);
  g.ld_gate = a.gate_stride, g.ld_up = a.up_stride, g.ld_dout = a.out_stride;
  g.pitch = 2 * p.slope_pitch;
  g.dgate = reinterpret_cast<uint16_t*>(ws + p.slopes), g.dup = g.dgate + p.slope_pitch;
  g.partial = p.sums >= 0 ? reinterpret_cast<float*>(ws + p.sums) : nullptr;
  g.M = a.rows, g.F = a.hidden, g.rows_per_block = (int)p.rows_per_block;
  e = f16 ? run_slopes<__half>(g, a.act, s) : run_slopes<__nv_bfloat16>(g, a.act, s);
  if (e != cudaSuccess) return e;
  // The products first: the sums that do not need them run while the last one ends.
  const int problems = (a.dw_gate ? 1 : 0) + (a.dw_up ? 1 : 0);
  Product dx{}, dw{};
  dx.f16 = dw.f16 = f16;
  if (a.dx) {
    Product& P = dx;
    if (p.partial >= 0) P.partial = reinterpret_cast<float*>(ws + p.partial);
    P.M = a.rows, P.N = a.width;
    P.k_half = (a.hidden + 63) / 64, P.k_blocks = 2 * P.k_half;
    P.splits = p.dx.splits;
    P.ldp = round_up(P.N, 4), P.plane = P.M * P.ldp;
    if (!operand_map(&P.a[0], 0, f16, g.dgate, a.hidden, a.rows, g.pitch, 128) ||
        !operand_map(&P.a[1], 0, f16, g.dup, a.hidden, a.rows, g.pitch, 128) ||
        !operand_map(&P.b[0], 0, f16, p.wg.p, a.width, a.hidden, p.wg.stride, 64) ||
        !operand_map(&P.b[1], 0, f16, p.wu.p, a.width, a.hidden, p.wu.stride, 64))
      return cudaErrorInvalidValue;
    output(P, 0, a.dx, a.dx_stride);
    e = run_product<DX, false>(P, p.dx, 1, s);
    if (e != cudaSuccess) return e;
  }
  if (problems) {
    Product& P = dw;
    if (p.partial_dw >= 0) P.partial = reinterpret_cast<float*>(ws + p.partial_dw);
    P.M = a.hidden, P.N = a.width;
    P.k_blocks = P.k_half = (int)((a.rows + 63) / 64);
    P.splits = p.dw.splits;
    P.ldp = round_up(P.N, 4), P.plane = P.M * P.ldp;
    int i = 0;
    if (a.dw_gate) {
      if (!operand_map(&P.a[i], 0, f16, g.dgate, a.hidden, a.rows, g.pitch, 64)) return cudaErrorInvalidValue;
      output(P, i++, a.dw_gate, a.dw_gate_stride);
    }
    if (a.dw_up) {
      if (!operand_map(&P.a[i], 0, f16, g.dup, a.hidden, a.rows, g.pitch, 64)) return cudaErrorInvalidValue;
      output(P, i++, a.dw_up, a.dw_up_stride);
    }
    if (!operand_map(&P.b[0], 0, f16, p.x.p, a.width, a.rows, p.x.stride, 64)) return cudaErrorInvalidValue;
    e = run_product<DW, false>(P, p.dw, problems, s);
    if (e == cudaSuccess && P.splits > 1) e = join<false>(P, problems, false, s);
    if (e != cudaSuccess) return e;
  }
  // dx's partial sums are complete where dW's product has begun
  if (a.dx && dx.splits > 1) e = join<false>(dx, 1, problems > 0, s);
  if (e == cudaSuccess && g.partial)
    e = column_sums(ColumnSums{g.partial, p.sum_blocks, 2 * p.slope_pitch, a.hidden, p.slope_pitch, {a.dbias_gate, a.dbias_up},
                               a.dx || problems}, s);
  return e;
}

}  // namespace

int64_t gated_ffn_workspace(const dit_gated_ffn_args& a, bool backward) {
  return a.rows == 0 ? 0 : make_plan(a, backward).bytes;
}
cudaError_t gated_ffn_run(const dit_gated_ffn_args& a, bool back, void* ws, cudaStream_t s) {
  if (!back && a.rows == 0) return cudaSuccess;
  return back ? backward(a, static_cast<char*>(ws), s) : forward(a, static_cast<char*>(ws), s);
}
cudaError_t gated_ffn_take_error(int* site, cudaStream_t s) {
  cudaError_t e = cudaStreamSynchronize(s);
  const int none = 0;
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(site, g_wait_error, sizeof(int));
  if (e == cudaSuccess && *site) e = cudaMemcpyToSymbol(g_wait_error, &none, sizeof(int));
  return e;
}

}  // namespace dit
