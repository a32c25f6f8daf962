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
  static constexpr int ESZ = F8 ? 1 : 2;
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
  int tma[3];           // output by tensor stores; else element by element
  float* partial;       // splits > 1: fp32 planes [problem][split][gate, up][M][ldp]
  int64_t ldp, plane;
  const float *x_scale, *scale[2], *bias[2];
  int64_t M;            // rows and columns of the output
  int N;
  int k_blocks, k_half; // DX: blocks of each half of K
  int m_tiles, n_tiles, group_n, splits, items;
  uint32_t idesc;
  int f16, act;
};

// ---------------------------------------------------------------- activation
// sigmoid(z) and 1 - sigmoid(z), each with a relative error of a few 2^-22
// (ex2.approx and rcp.approx; the results are rounded to 16 bits).
DIT_DEV float2 sigmoids(float z) {
  float e;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(-fabsf(z) * 1.4426950408889634f));
  const float r = __fdividef(1.f, 1.f + e);
  const float er = e * r;
  return z >= 0.f ? make_float2(r, er) : make_float2(er, r);
}
constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
DIT_DEV float activation(int act, float g) {
  const float z = act == DIT_ACT_SILU ? g : g * fmaf(kGelu2 * 0.044715f, g * g, kGelu2);
  return g * sigmoids(z).x;
}
// act(g) and act'(g)
DIT_DEV float2 activation_slope(int act, float g) {
  const float q = g * g;
  const float z = act == DIT_ACT_SILU ? g : g * fmaf(kGelu2 * 0.044715f, q, kGelu2);
  const float zp = act == DIT_ACT_SILU ? 1.f : fmaf(3.f * 0.044715f * kGelu2, q, kGelu2);
  const float2 s = sigmoids(z);
  // far out 1 - s is 0 and z' may be infinite: the limit of their product is 0
  return make_float2(g * s.x, s.x == 0.f || s.y == 0.f ? s.x : fmaf(g * s.x * s.y, zp, s.x));
}

DIT_DEV uint32_t pack16(int f16, float lo, float hi) { return f16 ? pack2<__half>(lo, hi) : pack_bf16x2(lo, hi); }

// Four values of a per-column array from column c on, 0 from n on.
DIT_DEV float4 columns4(const float* p, int c, int n, bool aligned) {
  if (aligned && c + 4 <= n) return __ldg(reinterpret_cast<const float4*>(p + c));
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < n) v.x = __ldg(p + c);
  if (c + 1 < n) v.y = __ldg(p + c + 1);
  if (c + 2 < n) v.z = __ldg(p + c + 2);
  if (c + 3 < n) v.w = __ldg(p + c + 3);
  return v;
}

// acc * (row_scale * scale) + bias over 32 columns
DIT_DEV void finish32(float (&v)[32], const Product& P, int side, float row_scale, int c0) {
  const float* sc = P.scale[side];
  const float* bi = P.bias[side];
  if (!sc && !bi) return;
  const bool sa = (reinterpret_cast<uintptr_t>(sc) & 15) == 0, ba = (reinterpret_cast<uintptr_t>(bi) & 15) == 0;
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const float4 b = bi ? columns4(bi, c0 + j, P.N, ba) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (sc) {
      const float4 w = columns4(sc, c0 + j, P.N, sa);
      v[j] = fmaf(v[j], row_scale * w.x, b.x), v[j + 1] = fmaf(v[j + 1], row_scale * w.y, b.y);
      v[j + 2] = fmaf(v[j + 2], row_scale * w.z, b.z), v[j + 3] = fmaf(v[j + 3], row_scale * w.w, b.w);
    } else {
      v[j] += b.x, v[j + 1] += b.y, v[j + 2] += b.z, v[j + 3] += b.w;
    }
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
DIT_DEV int split_begin(const Product& P, int z) { return (int)((int64_t)P.k_blocks * z / P.splits); }

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
  uint16_t* out = static_cast<uint16_t*>(P.out[o]);
  const int c = col0 + 2 * lane;
#pragma unroll 4
  for (int r = 0; r < 32 && row0 + r < P.M; ++r) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(stg + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
    uint16_t* at = out + (row0 + r) * P.ldo[o] + c;
    if (c < P.N) at[0] = (uint16_t)w;
    if (c + 1 < P.N) at[1] = (uint16_t)(w >> 16);
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
template <int MODE, int BN, class Release>
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
            finish32(g, P, 0, row_scale, col0 + hh * 32);
            finish32(v, P, 1, row_scale, col0 + hh * 32);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= activation(P.act, g[j]);
          } else {
            load32(at + (o - 1) * (BN / 2), v);
            wait32(v);
            finish32(v, P, o - 1, row_scale, col0 + hh * 32);
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

template <int MODE, bool F8, bool PAIR>
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
        const int kb1 = split_begin(P, t.z + 1);
        for (int kb = split_begin(P, t.z); kb < kb1; ++kb) {
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
        const Tile t = tile_of(P, item);
        const int kb0 = split_begin(P, t.z), kb1 = split_begin(P, t.z + 1);
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
      drain<MODE, C::BN>(P, t, tmem_base + acc * C::BN + ((uint32_t)(q * 32) << 16), row0, half, stg, release);
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
  float4 s = *reinterpret_cast<const float4*>(p);
#pragma unroll 4
  for (int z = 1; z < n; ++z) {
    const float4 t = *reinterpret_cast<const float4*>(p + z * step);
    s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
  }
  v[0] = s.x, v[1] = s.y, v[2] = s.z, v[3] = s.w;
}
// The splits of K joined in order, four columns a thread, then what the tile's
// epilogue would have done.  blockIdx.z: the problem.
template <bool GATED>
__global__ void __launch_bounds__(256) join_kernel(const Join J) {
  wait_previous();
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
        if (J.scale[0]) g[j] *= rs * __ldg(J.scale[0] + c + j), v[j] *= rs * __ldg(J.scale[1] + c + j);
        if (J.bias[0]) g[j] += __ldg(J.bias[0] + c + j);
        if (J.bias[1]) v[j] += __ldg(J.bias[1] + c + j);
      }
      if (J.out[1]) {
        store4(J.out[1], row * J.ldo[1] + c, n, J.f16, g);
        store4(J.out[2], row * J.ldo[2] + c, n, J.f16, v);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] *= activation(J.act, g[j]);
      store4(J.out[0], row * J.ldo[0] + c, n, J.f16, v);
    } else {
      sum_planes(p + (int64_t)blockIdx.z * J.splits * J.plane, J.plane, J.splits, v);
      store4(J.out[blockIdx.z], row * J.ldo[blockIdx.z] + c, n, J.f16, v);
    }
  }
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
  const int o = blockIdx.y;
  if (!a.src[o]) return;
  const E* src = reinterpret_cast<const E*>(a.src[o]);
  E* dst = reinterpret_cast<E*>(a.dst[o]);
  // a warp per row
  const int lane = threadIdx.x & 31;
  for (int64_t r = (blockIdx.x * 256ll + threadIdx.x) >> 5; r < a.rows[o]; r += gridDim.x * 8ll)
    for (int c = lane; c < a.width; c += 32) dst[r * a.pitch + c] = src[r * a.src_stride[o] + c];
}

// ---------------------------------------------------------------- gradients of gate and up
struct Slopes {
  const uint16_t *gate, *up, *dout;
  int64_t ld_gate, ld_up, ld_dout;
  uint16_t *dgate, *dup;  // at multiples of 16 bytes
  int64_t pitch;
  float* partial;         // [row block][2][pitch] sums of the block's rows, or NULL
  int64_t M;
  int F, rows_per_block, f16, act;
};

DIT_DEV void load8(const uint16_t* p, int n, int f16, float (&v)[8]) {
  uint32_t w[4];
  if (n >= 8 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    const uint4 t = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = (2 * j < n ? (uint32_t)p[2 * j] : 0u) | (2 * j + 1 < n ? (uint32_t)p[2 * j + 1] << 16 : 0u);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 t = f16 ? unpack2<__half>(w[j]) : unpack2<__nv_bfloat16>(w[j]);
    v[2 * j] = t.x, v[2 * j + 1] = t.y;
  }
}

// 256 columns (8 a lane) x rows_per_block rows a block, 8 rows at a time.
__global__ void __launch_bounds__(256) slopes_kernel(const Slopes a) {
  __shared__ float sums[8][2][32][9];
  wait_previous();
  const int lane = threadIdx.x, ty = threadIdx.y;
  const int c = (blockIdx.y * 32 + lane) * 8;
  const int n = a.F - c;
  float sg[8] = {}, su[8] = {};
  const int64_t r0 = (int64_t)blockIdx.x * a.rows_per_block;
  const int64_t r1 = min(a.M, r0 + a.rows_per_block);
  if (n > 0) {
    for (int64_t r = r0 + ty; r < r1; r += 8) {
      float g[8], u[8], d[8];
      load8(a.gate + r * a.ld_gate + c, n, a.f16, g);
      load8(a.up + r * a.ld_up + c, n, a.f16, u);
      load8(a.dout + r * a.ld_dout + c, n, a.f16, d);
      uint32_t wg[4], wu[4];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 s = activation_slope(a.act, g[j]);
        g[j] = d[j] * u[j] * s.y;
        u[j] = d[j] * s.x;
        if (j >= n) g[j] = u[j] = 0.f;
        sg[j] += g[j], su[j] += u[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        wg[j] = pack16(a.f16, g[2 * j], g[2 * j + 1]);
        wu[j] = pack16(a.f16, u[2 * j], u[2 * j + 1]);
      }
      // c + 8 <= pitch: the pitch is a multiple of 8
      *reinterpret_cast<uint4*>(a.dgate + r * a.pitch + c) = make_uint4(wg[0], wg[1], wg[2], wg[3]);
      *reinterpret_cast<uint4*>(a.dup + r * a.pitch + c) = make_uint4(wu[0], wu[1], wu[2], wu[3]);
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
Split choose(int64_t M, int64_t N, int64_t cols_per_n, int64_t k_blocks, int problems) {
  Split best{false, 1};
  double least = 0;
  for (int pair = 0; pair < 2; ++pair)
    for (int s = 1; s <= 16; ++s) {
      if (s > 1 && k_blocks / s < 4) break;
      const int64_t tm = pair ? 256 : 128, tn = (pair ? 256 : 128) / cols_per_n;
      const int64_t tiles = ((M + tm - 1) / tm) * ((N + tn - 1) / tn) * problems * s;
      const int64_t slots = pair ? kSms / 2 : kSms;
      double t = (double)((tiles + slots - 1) / slots) * (double)((k_blocks + s - 1) / s) * (pair ? 512. : 300.) + 4000.;
      if (s > 1) t += 5000. + (double)M * N * cols_per_n * problems * s * 8. / 3500.;
      if (least == 0 || t < least) least = t, best = Split{pair != 0, s};
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
  int64_t slopes = -1, slope_pitch = 0;   // [rows][2][pitch] 16-bit
  int64_t sums = -1, sum_blocks = 0, rows_per_block = 0;
  int64_t partial = -1;
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
  auto operand = [&](Operand& o, const void* ptr, int64_t stride, int64_t rows, bool used) {
    o.p = ptr, o.stride = stride;
    if (rows <= 1) o.stride = round_up(a.width, 16 / esz);  // the stride of a single row says nothing
    // as a tensor map wants them: 16-byte rows, strides below 2^40 bytes; rows that overlap are no matrix
    o.packed = used && ((((uintptr_t)ptr | (uintptr_t)(o.stride * esz)) & 15) != 0 || o.stride < a.width ||
                        o.stride * esz >= kMaxStride);
    o.pitch = round_up(a.width, 16 / esz);
    o.offset = o.packed ? p.take(rows * o.pitch * esz) : 0;
  };
  operand(p.x, a.x, a.x_stride, a.rows, !backward || a.dw_gate || a.dw_up);
  operand(p.wg, a.w_gate, a.w_gate_stride, a.hidden, !backward || a.dx);
  operand(p.wu, a.w_up, a.w_up_stride, a.hidden, !backward || a.dx);
  const int bk = 128 / esz;
  if (!backward) {
    p.fwd = choose(a.rows, a.hidden, 2, (a.width + bk - 1) / bk, 1);
    if (p.fwd.splits > 1) p.partial = p.take(planes(p.fwd, a.rows, a.hidden, 2));
    return p;
  }
  p.slope_pitch = round_up(a.hidden, 8);
  p.slopes = p.take(a.rows * p.slope_pitch * 2 * 2);
  // few rows a block while there are few blocks; at most 32 serial additions either way
  p.rows_per_block = a.rows * a.hidden > (1 << 24) ? 256 : 32;
  p.sum_blocks = (a.rows + p.rows_per_block - 1) / p.rows_per_block;
  if (a.dbias_gate || a.dbias_up) p.sums = p.take(p.sum_blocks * 2 * p.slope_pitch * 4);
  const int problems = (a.dw_gate ? 1 : 0) + (a.dw_up ? 1 : 0);
  int64_t most = 0;
  if (a.dx) {
    p.dx = choose(a.rows, a.width, 1, 2 * ((a.hidden + 63) / 64), 1);
    most = planes(p.dx, a.rows, a.width, 1);
  }
  if (problems) {
    p.dw = choose(a.hidden, a.width, 1, (a.rows + 63) / 64, problems);
    const int64_t n = planes(p.dw, a.hidden, a.width, problems);
    most = n > most ? n : most;
  }
  if (most) p.partial = p.take(most);
  return p;
}

// ---------------------------------------------------------------- launches
// CTAs, or pairs of them, that run at once on the current device: a persistent
// launch asks for no more (one that had to wait would run its whole share last).
template <int MODE, bool F8, bool PAIR>
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
      const auto kernel = product_kernel<MODE, F8, PAIR>;
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

template <int MODE, bool F8, bool PAIR>
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
  const cudaError_t e = resident<MODE, F8, PAIR>(&slots);
  if (e != cudaSuccess) return e;
  const int n = P.items < slots ? P.items : slots;
  return launch_kernel(product_kernel<MODE, F8, PAIR>, dim3(PAIR ? 2 * n : n), dim3(kThreads), C::SMEM, s, PAIR ? 2 : 1, true, P);
}
template <int MODE, bool F8>
cudaError_t run_product(Product& P, const Split& sp, int problems, cudaStream_t s) {
  P.splits = sp.splits;
  return sp.pair ? launch_product<MODE, F8, true>(P, problems, s) : launch_product<MODE, F8, false>(P, problems, s);
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
cudaError_t join(const Product& P, int problems, cudaStream_t s) {
  Join J{P.partial, P.ldp, P.plane, P.splits, P.x_scale, {P.scale[0], P.scale[1]}, {P.bias[0], P.bias[1]},
         {P.out[0], P.out[1], P.out[2]}, {P.ldo[0], P.ldo[1], P.ldo[2]}, P.M, P.N, P.f16, P.act};
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

cudaError_t forward(const dit_gated_ffn_args& a, char* ws, cudaStream_t s) {
  Plan p = make_plan(a, false);
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
  return e != cudaSuccess || P.splits == 1 ? e : join<true>(P, 1, s);
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
  g.M = a.rows, g.F = a.hidden, g.rows_per_block = (int)p.rows_per_block, g.f16 = f16, g.act = a.act;
  e = launch_kernel(slopes_kernel, dim3((unsigned)p.sum_blocks, (unsigned)((a.hidden + 255) / 256)), dim3(32, 8), 0, s, 1, false, g);
  if (e != cudaSuccess) return e;
  if (g.partial) {
    ColumnSums c{g.partial, p.sum_blocks, 2 * p.slope_pitch, a.hidden, p.slope_pitch, {a.dbias_gate, a.dbias_up}};
    e = launch_kernel(column_sums_kernel<0>, dim3((a.hidden + 31) / 32, 2), dim3(32, 32), 0, s, 1, false, c);
    if (e != cudaSuccess) return e;
  }
  Product P{};
  P.f16 = f16;
  if (p.partial >= 0) P.partial = reinterpret_cast<float*>(ws + p.partial);
  if (a.dx) {
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
    if (e == cudaSuccess && P.splits > 1) e = join<false>(P, 1, s);
    if (e != cudaSuccess) return e;
  }
  if (a.dw_gate || a.dw_up) {
    const int problems = (a.dw_gate ? 1 : 0) + (a.dw_up ? 1 : 0);
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
    if (e == cudaSuccess && P.splits > 1) e = join<false>(P, problems, s);
  }
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
