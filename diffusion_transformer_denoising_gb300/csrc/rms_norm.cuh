// RMS norm over channels with the residual's addition in front of it, into the
// activations' type or into e4m3 with a scale for each row, and its gradient.
//
// Mathematics.  v = x + residual rounded to the type, r = (mean v^2 + eps)^-1/2,
// y = v r w, in this order: v w may vanish or overflow where v r, of size 1, does not.
// e4m3: scale = max |y| / 448, y / scale rounded to nearest even.
// Gradient: g = dy w, dx = dtotal + r (g - v r^2 mean(g v)), dw = sum dy v r: the two
// row sums (v^2 and g v) are taken together.
//
// What bounds it: HBM.  Every row is read once and written once.  A forward row of
// whole 16-byte vectors is held in registers, by 1 to 16 warps.  The gradient holds
// two or three tensors' rows and the weight's sums, too much for enough warps, so its
// rows come through a ring in shared memory that asynchronous copies fill: while a
// row is worked on the next is on its way, whatever the registers hold.  So do rows
// of any other alignment, which are read and written through shifted windows.  Narrow
// rows share a warp.
//
// Measured on one GB300 (bf16, 1536 channels, device time): 2 x 32760 rows with a
// residual 112 us = 7.2 TB/s; 32760 into e4m3 54 us = 6.5 TB/s; their gradient 66 us =
// 6.1 TB/s and 5 us for the weight's sums.  68311 odd rows of 1535: 173 us (floor 124),
// gradient 240 (124).
#pragma once
#include <math.h>

#include "column_sums.cuh"
#include "launch.cuh"
#include "operators.h"
#include "vec.cuh"

namespace dit {

namespace norm {

enum NormMode { SAME, E4M3, GRAD };
enum { AL_X = 1, AL_RES = 2, AL_TOTAL = 4, AL_DY = 8, AL_OUT = 16, AL_W = 32 };

struct Norm {
  const void *x, *res, *dy;
  void *total, *out;
  int64_t sx[2], sres[2], stotal[2], sdy[2], sout[2];
  float* scale;
  const float* w;
  float* partial;  // GRAD: [block][channels] sums of the block's rows, or NULL
  uint32_t rows, tokens;
  int C;
  float eps;
  int aligned;     // AL_*: 16-byte rows (AL_OUT of e4m3: 8-byte rows for chunks of 8, 4 for 4)
  bool words;      // 16-bit rows of 4-byte words, not all of them of 16-byte vectors
};

// max(a, |b|, |c|), NaN if one of them is
DIT_DEV float max_abs(float a, float2 b) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b.x), "f"(b.y));
  return d;
}
DIT_DEV float rcp_approx(float x) {  // within 2^-23
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
DIT_DEV float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// What an e4m3 row is held in: top is max |y|.  v r comes before the weight: v w of a row of
// 1e-37 has lost digits that y (of 1e-34 at eps 1e-6) has, and r over its scale is infinite.
struct RowScale {
  float scale, factor;  // out = y factor
  bool finite;
};
DIT_DEV RowScale row_scale(float top) {
  RowScale q;
  q.finite = top <= 3.402823466e38f;
  // below 448 x 2^-126 the scale stays a normal number, so that its reciprocal is finite
  q.scale = !q.finite ? __int_as_float(0x7fffffff) : top > 0.f ? fmaxf(top / kE4M3Max, 1.17549435e-38f) : 1.f;
  q.factor = q.finite ? rcp_approx(q.scale) : 0.f;
  return q;
}

// A 16-byte chunk's values as pairs, for the packed fp32 instructions (the first
// kernels' scalar ones took the gradient of the video case 104 us).
template <typename T>
struct Pairs {
  static constexpr int E = 16 / sizeof(T), N = E / 2;
  float2 v[N];
  DIT_DEV float2& operator[](int j) { return v[j]; }
  DIT_DEV const float2& operator[](int j) const { return v[j]; }
};
template <typename T>
DIT_DEV Pairs<T> pairs(const uint4& r) {
  Pairs<T> p;
  const uint32_t* w = &r.x;
#pragma unroll
  for (int j = 0; j < Pairs<T>::N; ++j) {
    if constexpr (sizeof(T) == 4) p[j] = make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    else p[j] = unpack2<T>(w[j]);
  }
  return p;
}
template <typename T>
DIT_DEV uint4 packed(const Pairs<T>& p) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(p[0].x), __float_as_uint(p[0].y), __float_as_uint(p[1].x), __float_as_uint(p[1].y));
  else
    return make_uint4(pack2<T>(p[0].x, p[0].y), pack2<T>(p[1].x, p[1].y), pack2<T>(p[2].x, p[2].y), pack2<T>(p[3].x, p[3].y));
}

// The chunk at p, of which n elements are there (zeros behind them).  WORDS: rows of
// 4-byte words, which go two 16-bit elements at a time.
template <typename T, bool WHOLE, bool WORDS = false>
DIT_DEV uint4 load_chunk(const T* p, int n, bool aligned) {
  constexpr int E = 16 / sizeof(T);
  if (WHOLE || (aligned && n >= E)) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4] = {0, 0, 0, 0};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < n) w[j] = reinterpret_cast<const uint32_t*>(p)[j];
  } else if constexpr (WORDS) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (2 * j + 1 < n) w[j] = reinterpret_cast<const uint32_t*>(p)[j];
      else if (2 * j < n) w[j] = q[2 * j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < n) w[j / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[j] << (16 * (j & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T, bool WHOLE, bool WORDS = false>
DIT_DEV void store_chunk(T* p, int n, bool aligned, const uint4& r) {
  constexpr int E = 16 / sizeof(T);
  if (WHOLE || (aligned && n >= E)) {
    *reinterpret_cast<uint4*>(p) = r;
    return;
  }
  const uint32_t* w = &r.x;
  if constexpr (WORDS) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (2 * j + 1 < n) reinterpret_cast<uint32_t*>(p)[j] = w[j];
      else if (2 * j < n) reinterpret_cast<uint16_t*>(p)[2 * j] = (uint16_t)w[j];
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < E; ++j) {
    if (j >= n) continue;
    if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(p)[j] = w[j];
    else reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
  }
}
template <typename T, bool WHOLE>
DIT_DEV void store_e4m3(uint8_t* p, int n, bool aligned, const Pairs<T>& v) {
  constexpr int E = 16 / sizeof(T);
  uint32_t w[E / 4];
#pragma unroll
  for (int j = 0; j < E / 4; ++j) w[j] = pack_e4m3x4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
  if (WHOLE || (aligned && n >= E)) {
    if constexpr (E == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
    return;
  }
#pragma unroll
  for (int j = 0; j < E; ++j)
    if (j < n) p[j] = (uint8_t)(w[j / 4] >> (8 * (j & 3)));
}
// v *= the weights of channels c on (zeros behind the last; WHOLE: n is E or, behind the
// row's end, not above 0).  Only the load stands under that condition: a branch around the
// products or an index held to the last weights took the video pair 145 us, this 118.
template <typename T, bool WHOLE>
DIT_DEV void times_weight(Pairs<T>& v, const float* w, int c, int n, bool aligned) {
  constexpr int E = 16 / sizeof(T);
  if (!WHOLE && !w) return;
  if (WHOLE || (aligned && n >= E)) {
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!WHOLE || n > 0) t = __ldg(reinterpret_cast<const float4*>(w + c + j));
      v[j / 2] = fmul2(v[j / 2], make_float2(t.x, t.y));
      v[j / 2 + 1] = fmul2(v[j / 2 + 1], make_float2(t.z, t.w));
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; j += 2)
      v[j / 2] = fmul2(v[j / 2], make_float2(j < n ? __ldg(w + c + j) : 0.f, j + 1 < n ? __ldg(w + c + j + 1) : 0.f));
  }
}
template <typename T>
DIT_DEV void scale_by(Pairs<T>& v, float k) {
#pragma unroll
  for (int j = 0; j < Pairs<T>::N; ++j) v[j] = fmul2(v[j], make_float2(k, k));
}
// sum += a b, pair by pair
template <typename T>
DIT_DEV void add_products(float2& sum, const Pairs<T>& a, const Pairs<T>& b) {
#pragma unroll
  for (int j = 0; j < Pairs<T>::N; ++j) sum = ffma2(a[j], b[j], sum);
}
template <typename T>
DIT_DEV void add_to(Pairs<T>& a, const Pairs<T>& b) {
#pragma unroll
  for (int j = 0; j < Pairs<T>::N; ++j) a[j] = fadd2(a[j], b[j]);
}
// g = dy, gw = dy w and v of a chunk: dw += g v r, gw becomes r (gw - k v)
template <typename T>
DIT_DEV void norm_gradient(const Pairs<T>& g, Pairs<T>& gw, const Pairs<T>& v, float r, float k, Pairs<T>& dw) {
  const float2 r2 = make_float2(r, r), k2 = make_float2(-k, -k);
#pragma unroll
  for (int j = 0; j < Pairs<T>::N; ++j) {
    dw[j] = ffma2(g[j], fmul2(v[j], r2), dw[j]);
    gw[j] = fmul2(r2, ffma2(k2, v[j], gw[j]));
  }
}

DIT_DEV float2 warp_sum2(float2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fadd2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  return v;
}
DIT_DEV float warp_sum1(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
DIT_DEV float warp_max1(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Asynchronous copy of 16 bytes, of which `bytes` are there, zeros behind them.
DIT_DEV void copy_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
DIT_DEV void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
DIT_DEV void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

constexpr int kRingStages = 2;
// RW warps hold a row, NV chunks of 16 bytes a thread; ROWS rows a block.
template <int RW, int NV, int ROWS, int MODE, bool RES, bool WHOLE>
struct Ring {
  static constexpr int INPUTS = (MODE == GRAD ? 2 : 1) + (RES ? 1 : 0);
  static constexpr int ROW = RW * NV * 512;            // bytes
  static constexpr int SLOT = ROW + (WHOLE ? 0 : 16);  // a row that begins inside a vector
  static constexpr int STAGE = INPUTS * SLOT;
  static constexpr int SMEM = ROWS * kRingStages * STAGE;
};
// Blocks of a ring kernel that an SM holds (registers allow them too: launch bounds).
// `held`: the gradient of rows that are not whole keeps them in registers, and fewer
// warps have room (with 24 of them, three chunks a thread spilled: 317 us instead of
// 240 for 68311 rows of 1535 bf16 channels; two gain: 180 and 197 us for 52376 of 1001 in fp32).
constexpr int ring_blocks(int rw, int nv, int rows, int inputs, bool held) {
  const int n = (227 << 10) / (rows * kRingStages * inputs * (rw * nv * 512 + 16) + 1024);
  int most = (nv >= 4 || (rw == 1 && nv > 1) || (held && nv == 3) ? 16 : held && nv > 1 ? 24 : 32) / (rw * rows);
  if (most < 1) most = 1;
  return n > most ? most : n;
}

// The warps of a row wait for each other.
template <int RW>
DIT_DEV void row_sync() {
  if constexpr (RW == 1) __syncwarp();
  else named_bar_sync(1 + threadIdx.x / (32 * RW), 32 * RW);
}

// A row of 16-byte vectors into a slot of shared memory, zeros up to its last chunk's
// end: each thread fetches the chunks that it reads.
template <int RW, int NV>
DIT_DEV void fetch_vectors(uint8_t* slot, const uint8_t* src, int bytes) {
  const int lane = threadIdx.x & (32 * RW - 1);
  const uint32_t dst = smem_u32(slot);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (lane + 32 * RW * i) * 16;
    if (at < bytes) copy_async16(dst + at, src + at, min(16, bytes - at));
  }
}
// A row of any alignment into a slot, at the place in its first vector that it has in
// memory: the vectors between its ends by asynchronous copies, each byte of the
// vectors that it shares with its neighbours by a load of its own, which is put into
// the slot when the row's turn comes.  (Copies of 4 and loads of 2 bytes for the whole
// row took 234 us for 68311 rows of 1535 bf16 channels, 326 us for the gradient.)
struct Edge {
  uint32_t value;
  int at;  // byte of the slot, -1: none
};
template <int RW>
DIT_DEV Edge fetch_bytes(uint8_t* slot, const uint8_t* src, int bytes) {
  const int lane = threadIdx.x & (32 * RW - 1), o = (int)(reinterpret_cast<uintptr_t>(src) & 15);
  const uint8_t* base = src - o;
  const int first = o ? 1 : 0, end = (o + bytes) >> 4;
  const uint32_t dst = smem_u32(slot);
  for (int v = first + lane; v < end; v += 32 * RW) copy_async16(dst + v * 16, base + v * 16, 16);
  Edge e{0, -1};
  if (o && lane < min(16 - o, bytes)) e.at = o + lane;
  const int tail = max(first, end) * 16;  // a row inside one vector has no tail
  if (lane >= 16 && lane - 16 < o + bytes - tail && lane < 32) e.at = tail + lane - 16;
  if (e.at >= 0) e.value = base[e.at];
  return e;
}
// 16 bytes from byte at + s of a slot on (at a multiple of 16, s < 16 the same for the row).
DIT_DEV uint4 window(const uint8_t* slot, int at, int s) {
  const uint4 a = *reinterpret_cast<const uint4*>(slot + at);
  return s == 0 ? a : shift16(a, *reinterpret_cast<const uint4*>(slot + at + 16), s);
}
// The first n elements of a chunk, zeros behind them.
template <typename T>
DIT_DEV uint4 first_of(uint4 r, int n) {
  constexpr int E = 16 / sizeof(T);
  if (n >= E) return r;
  uint32_t* w = &r.x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 4) w[j] = j < n ? w[j] : 0u;
    else w[j] = 2 * j + 1 < n ? w[j] : 2 * j < n ? w[j] & 0xffffu : 0u;
  }
  return r;
}
// A row that lies from a slot's begin on, out to memory of any alignment.
template <int RW>
DIT_DEV void put_bytes(uint8_t* dst, const uint8_t* slot, int bytes) {
  const int lane = threadIdx.x & (32 * RW - 1), o = (int)(reinterpret_cast<uintptr_t>(dst) & 15);
  uint8_t* base = dst - o;
  const int first = o ? 1 : 0, end = (o + bytes) >> 4;
  for (int v = first + lane; v < end; v += 32 * RW) *reinterpret_cast<uint4*>(base + v * 16) = window(slot, (v - first) * 16, (16 - o) & 15);
  int at = -1;
  if (o && lane < min(16 - o, bytes)) at = o + lane;
  const int tail = max(first, end) * 16;
  if (lane >= 16 && lane - 16 < o + bytes - tail && lane < 32) at = tail + lane - 16;
  if (at >= 0) base[at] = slot[at - o];
}

// RW warps a row, NV chunks of 16 bytes a thread: chunk lane + 32 RW i.  WHOLE: a weight,
// every tensor in rows of whole 16-byte vectors (no branch is left in a row then, and
// its loads are issued together: the video gradient 90 us without it).
template <typename T, int RW, int NV, int ROWS, int MODE, bool RES, bool WHOLE>
__global__ void __launch_bounds__(32 * RW * ROWS, ring_blocks(RW, NV, ROWS, Ring<RW, NV, ROWS, MODE, RES, WHOLE>::INPUTS, MODE == GRAD && !WHOLE))
    norm_ring_kernel(const Norm a) {
  constexpr int E = 16 / sizeof(T), TPR = 32 * RW;
  using R = Ring<RW, NV, ROWS, MODE, RES, WHOLE>;
  extern __shared__ uint4 ring_smem[];  // the ring; of several warps a row, their sums behind it
  const int lane = threadIdx.x & (TPR - 1), mine_row = threadIdx.x / TPR;
  uint8_t* const mine = reinterpret_cast<uint8_t*>(ring_smem) + mine_row * kRingStages * R::STAGE;
  const uint32_t step = gridDim.x * ROWS;
  float2* const parts = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(ring_smem) + R::SMEM) + mine_row * 2 * RW;
  int turn = 0;
  auto row_sum = [&](float2 v) {
    v = MODE == GRAD ? warp_sum2(v) : make_float2(warp_sum1(v.x), 0.f);
    if constexpr (RW > 1) {
      if ((lane & 31) == 0) parts[turn * RW + (lane >> 5)] = v;
      row_sync<RW>();
      v = parts[turn * RW];
#pragma unroll
      for (int i = 1; i < RW; ++i) v = fadd2(v, parts[turn * RW + i]);
      turn ^= 1;
    }
    return v;
  };
  auto row_max = [&](float v) {
    v = warp_max1(v);
    if constexpr (RW > 1) {
      if ((lane & 31) == 0) parts[turn * RW + (lane >> 5)].x = v;
      row_sync<RW>();
      v = parts[turn * RW].x;
#pragma unroll
      for (int i = 1; i < RW; ++i) v = max_nan(v, parts[turn * RW + i].x);
      turn ^= 1;
    }
    return v;
  };
  const int C = a.C, bytes = C * (int)sizeof(T);
  const float inv_c = 1.f / (float)C;
  auto offset = [&](uint32_t row, const int64_t (&s)[2]) {
    const uint32_t b = row / a.tokens;
    return (int64_t)b * s[0] + (int64_t)(row - b * a.tokens) * s[1];
  };
  // inputs 0: x, then dy, then residual; where each row begins in its first vector
  constexpr int RESIDUAL = R::INPUTS - 1;
  Edge edge[R::INPUTS], next_edge[R::INPUTS];
  int begin[R::INPUTS], next_begin[R::INPUTS];
#pragma unroll
  for (int i = 0; i < R::INPUTS; ++i) edge[i].at = next_edge[i].at = -1, begin[i] = next_begin[i] = 0;
  auto fetch_one = [&](int i, uint8_t* slot, const T* p, int flag) {
    const uint8_t* src = reinterpret_cast<const uint8_t*>(p);
    if (WHOLE || (a.aligned & flag)) {
      fetch_vectors<RW, NV>(slot + i * R::SLOT, src, bytes);
    } else {
      next_edge[i] = fetch_bytes<RW>(slot + i * R::SLOT, src, bytes);
      next_begin[i] = (int)(reinterpret_cast<uintptr_t>(src) & 15);
    }
  };
  auto fetch = [&](int stage, uint32_t row) {
    uint8_t* slot = mine + stage * R::STAGE;
    fetch_one(0, slot, static_cast<const T*>(a.x) + offset(row, a.sx), AL_X);
    if constexpr (MODE == GRAD) fetch_one(1, slot, static_cast<const T*>(a.dy) + offset(row, a.sdy), AL_DY);
    if constexpr (RES) fetch_one(RESIDUAL, slot, static_cast<const T*>(a.res) + offset(row, a.sres), AL_RES);
  };
  Pairs<T> dw[MODE == GRAD ? NV : 1] = {};
  uint32_t row = blockIdx.x * ROWS + mine_row;
  if (row < a.rows) fetch(0, row);
  copy_commit();
  int stage = 0;
  for (; row < a.rows; row += step, stage ^= 1) {
    uint8_t* const slot = mine + stage * R::STAGE;
    if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < R::INPUTS; ++i) edge[i] = next_edge[i], begin[i] = next_begin[i];
    }
    const bool more = step < a.rows - row;
    if (more) fetch(stage ^ 1, row + step);
    copy_commit();
    copy_wait<1>();
    if constexpr (!WHOLE) {  // (WHOLE: a thread reads what it has fetched)
#pragma unroll
      for (int i = 0; i < R::INPUTS; ++i)
        if (edge[i].at >= 0) slot[i * R::SLOT + edge[i].at] = (uint8_t)edge[i].value;
      row_sync<RW>();
    }
    // the chunk of channels c .. c + n of an input's row
    auto chunk = [&](int input, int i, int n) {
      const uint8_t* s = slot + input * R::SLOT;
      const int at = (lane + TPR * i) * 16;
      if constexpr (WHOLE) return *reinterpret_cast<const uint4*>(s + at);
      else return first_of<T>(window(s, at, begin[input]), n);
    };
    // results that are not stored as vectors go out through a slot, from its begin on
    auto put = [&](int input, int i) -> uint4& { return *reinterpret_cast<uint4*>(slot + input * R::SLOT + (lane + TPR * i) * 16); };
    const bool direct = WHOLE || (a.aligned & AL_OUT);
    if constexpr (MODE == GRAD) {
      float2 square = make_float2(0.f, 0.f), dot = square;
      uint4 x_held[WHOLE ? 1 : NV], dy_held[WHOLE ? 1 : NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + TPR * i) * E, n = WHOLE ? (C - c > 0 ? E : 0) : C - c;
        if (n <= 0) continue;
        const uint4 x_raw = chunk(0, i, n), dy_raw = chunk(1, i, n);
        if constexpr (!WHOLE) x_held[i] = x_raw, dy_held[i] = dy_raw;
        const Pairs<T> v = pairs<T>(x_raw);
        Pairs<T> g = pairs<T>(dy_raw);
        times_weight<T, WHOLE>(g, a.w, c, n, a.aligned & AL_W);
        add_products<T>(square, v, v);
        add_products<T>(dot, g, v);
      }
      const float2 sums = row_sum(make_float2(square.x + square.y, dot.x + dot.y));
      const float r = rsqrtf(fmaf(sums.x, inv_c, a.eps)), k = r * r * (sums.y * inv_c);
      T* out = static_cast<T*>(a.out) + offset(row, a.sout);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + TPR * i) * E, n = WHOLE ? (C - c > 0 ? E : 0) : C - c;
        if (n <= 0) continue;
        const Pairs<T> v = pairs<T>(WHOLE ? chunk(0, i, n) : x_held[WHOLE ? 0 : i]);
        const Pairs<T> g = pairs<T>(WHOLE ? chunk(1, i, n) : dy_held[WHOLE ? 0 : i]);
        Pairs<T> d = g;
        times_weight<T, WHOLE>(d, a.w, c, n, a.aligned & AL_W);
        norm_gradient<T>(g, d, v, r, k, dw[i]);
        if constexpr (RES) add_to<T>(d, pairs<T>(chunk(RESIDUAL, i, n)));
        if (direct) store_chunk<T, WHOLE>(out + c, n, true, packed<T>(d));
        else x_held[WHOLE ? 0 : i] = packed<T>(d);
      }
      if constexpr (!WHOLE) {
        if (!direct) {
          row_sync<RW>();  // the row's windows have been read
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if ((lane + TPR * i) * E < C) put(0, i) = x_held[i];
          row_sync<RW>();
          put_bytes<RW>(reinterpret_cast<uint8_t*>(out), slot, bytes);
        }
      }
    } else {
      Pairs<T> v[NV];
      float2 square = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + TPR * i) * E, n = WHOLE ? (C - c > 0 ? E : 0) : C - c;
        v[i] = Pairs<T>{};
        if (n <= 0) continue;
        v[i] = pairs<T>(chunk(0, i, n));
        if constexpr (RES) {
          add_to<T>(v[i], pairs<T>(chunk(RESIDUAL, i, n)));
          const uint4 sum = packed<T>(v[i]);
          v[i] = pairs<T>(sum);  // the norm is of the sum as it is kept
          if (a.total && (a.aligned & AL_TOTAL)) store_chunk<T, WHOLE>(static_cast<T*>(a.total) + offset(row, a.stotal) + c, n, true, sum);
        }
        add_products<T>(square, v[i], v[i]);
      }
      const float r = rsqrtf(fmaf(row_sum(make_float2(square.x + square.y, 0.f)).x, inv_c, a.eps));
      const bool put_total = RES && a.total && !(a.aligned & AL_TOTAL);
      if (put_total || !direct) {
        row_sync<RW>();  // the row's windows have been read
        if (put_total) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if ((lane + TPR * i) * E < C) put(0, i) = packed<T>(v[i]);  // exact: v is of the type
          row_sync<RW>();
          put_bytes<RW>(reinterpret_cast<uint8_t*>(static_cast<T*>(a.total) + offset(row, a.stotal)), slot, bytes);
          if (RESIDUAL == 0) row_sync<RW>();
        }
      }
      float factor = 1.f, top = 0.f;
      bool finite = true;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + TPR * i) * E, n = WHOLE ? (C - c > 0 ? E : 0) : C - c;
        if (n <= 0) continue;
        scale_by<T>(v[i], r);
        times_weight<T, WHOLE>(v[i], a.w, c, n, a.aligned & AL_W);
        if constexpr (MODE == E4M3)
#pragma unroll
          for (int j = 0; j < Pairs<T>::N; ++j) top = max_abs(top, v[i][j]);
      }
      if constexpr (MODE == E4M3) {
        const RowScale q = row_scale(row_max(top));
        factor = q.factor, finite = q.finite;
        if (lane == 0) a.scale[row] = q.scale;
      }
      T* out = static_cast<T*>(a.out) + offset(row, a.sout);
      uint8_t* out8 = static_cast<uint8_t*>(a.out) + offset(row, a.sout);
      uint8_t* const out_slot = slot + RESIDUAL * R::SLOT;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + TPR * i) * E, n = WHOLE ? (C - c > 0 ? E : 0) : C - c;
        if (n <= 0) continue;
        if constexpr (MODE == E4M3) {
          scale_by<T>(v[i], factor);
          const Pairs<T> q = finite ? v[i] : Pairs<T>{};
          if (direct) store_e4m3<T, WHOLE>(out8 + c, n, true, q);
          else store_e4m3<T, true>(out_slot + c, E, true, q);
        } else if (direct) {
          store_chunk<T, WHOLE>(out + c, n, true, packed<T>(v[i]));
        } else {
          put(RESIDUAL, i) = packed<T>(v[i]);
        }
      }
      if (!direct) {
        row_sync<RW>();
        put_bytes<RW>(MODE == E4M3 ? out8 : reinterpret_cast<uint8_t*>(out), out_slot, MODE == E4M3 ? C : bytes);
      }
    }
    if constexpr (!WHOLE) row_sync<RW>();  // the slot may be filled again
    if (!more) break;  // row + step may pass 32 bits
  }
  if constexpr (MODE == GRAD) {
    if (!a.partial) return;
    // the sums of the block's rows, through the ring
    copy_wait<0>();
    __syncthreads();
    float* join = reinterpret_cast<float*>(ring_smem);  // [row][channel]
    constexpr int WIDTH = NV * TPR * E;
    static_assert(ROWS * WIDTH * 4 <= R::SMEM, "room for the join");
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < E / 2; j += 2)
        *reinterpret_cast<float4*>(join + mine_row * WIDTH + (lane + TPR * i) * E + 2 * j) = make_float4(dw[i][j].x, dw[i][j].y, dw[i][j + 1].x, dw[i][j + 1].y);
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += TPR * ROWS) {
      float s = join[c];
#pragma unroll
      for (int g = 1; g < ROWS; ++g) s += join[g * WIDTH + c];
      a.partial[(int64_t)blockIdx.x * C + c] = s;
    }
  }
}

// Narrow rows: LPR lanes hold a row, a chunk each, 32 / LPR rows a warp, kNarrowBatch
// of such groups of rows under way at once.  (A warp a row took 375 us for 1.6 M rows
// of 64 bf16 channels, 493 us for the gradient.)  WORDS is a form of its own: with the
// choice made at each chunk rows that are not of words took 570 us instead of 466.
// Rows of words: 1.34 M of 78 channels 223 us, 449 by elements; gradients 289 and 721.
constexpr int kNarrowWarps = 4, kNarrowBatch = 4;
template <typename T, int LPR, int MODE, bool WORDS>
__global__ void __launch_bounds__(32 * kNarrowWarps) norm_narrow_kernel(const Norm a) {
  constexpr int E = 16 / sizeof(T), RPW = 32 / LPR, U = kNarrowBatch;
  __shared__ float join[MODE == GRAD ? kNarrowWarps : 1][LPR * E];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (lane % LPR) * E, n = a.C - c;
  const float inv_c = 1.f / (float)a.C;
  Pairs<T> w, dw = {};
#pragma unroll
  for (int j = 0; j < Pairs<T>::N; ++j) w[j] = make_float2(1.f, 1.f);
  times_weight<T, false>(w, a.w, c, n, false);
  auto row_sum = [](float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  const int64_t step = (int64_t)gridDim.x * kNarrowWarps * RPW * U;
  for (int64_t base = ((int64_t)blockIdx.x * kNarrowWarps + warp) * RPW * U; base < a.rows; base += step) {
    uint4 x[U], res[U], dy[MODE == GRAD ? U : 1];
    uint32_t b[U], t[U];
    bool there[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = base + u * RPW + lane / LPR;
      there[u] = row < a.rows && n > 0;
      b[u] = (uint32_t)row / a.tokens, t[u] = (uint32_t)row - b[u] * a.tokens;
      x[u] = res[u] = make_uint4(0, 0, 0, 0);
      if constexpr (MODE == GRAD) dy[u] = make_uint4(0, 0, 0, 0);
      if (!there[u]) continue;
      x[u] = load_chunk<T, false, WORDS>(static_cast<const T*>(a.x) + b[u] * a.sx[0] + t[u] * a.sx[1] + c, n, a.aligned & AL_X);
      if (a.res) res[u] = load_chunk<T, false, WORDS>(static_cast<const T*>(a.res) + b[u] * a.sres[0] + t[u] * a.sres[1] + c, n, a.aligned & AL_RES);
      if constexpr (MODE == GRAD) dy[u] = load_chunk<T, false, WORDS>(static_cast<const T*>(a.dy) + b[u] * a.sdy[0] + t[u] * a.sdy[1] + c, n, a.aligned & AL_DY);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Pairs<T> v = pairs<T>(x[u]);
      const int64_t at_out = b[u] * a.sout[0] + t[u] * a.sout[1] + c;
      float2 square = make_float2(0.f, 0.f);
      if constexpr (MODE == GRAD) {
        const Pairs<T> g = pairs<T>(dy[u]);
        Pairs<T> d = g;
        float2 dot = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < Pairs<T>::N; ++j) d[j] = fmul2(d[j], w[j]);
        add_products<T>(square, v, v);
        add_products<T>(dot, d, v);
        const float r = rsqrtf(fmaf(row_sum(square.x + square.y), inv_c, a.eps)), k = r * r * (row_sum(dot.x + dot.y) * inv_c);
        if (!there[u]) continue;
        norm_gradient<T>(g, d, v, r, k, dw);
        if (a.res) add_to<T>(d, pairs<T>(res[u]));
        store_chunk<T, false, WORDS>(static_cast<T*>(a.out) + at_out, n, a.aligned & AL_OUT, packed<T>(d));
      } else {
        if (a.res) {
          add_to<T>(v, pairs<T>(res[u]));
          const uint4 sum = packed<T>(v);
          v = pairs<T>(sum);  // the norm is of the sum as it is kept
          if (a.total && there[u]) store_chunk<T, false, WORDS>(static_cast<T*>(a.total) + b[u] * a.stotal[0] + t[u] * a.stotal[1] + c, n, a.aligned & AL_TOTAL, sum);
        }
        add_products<T>(square, v, v);
        const float r = rsqrtf(fmaf(row_sum(square.x + square.y), inv_c, a.eps));
        scale_by<T>(v, r);
#pragma unroll
        for (int j = 0; j < Pairs<T>::N; ++j) v[j] = fmul2(v[j], w[j]);
        if constexpr (MODE == E4M3) {
          float top = 0.f;
#pragma unroll
          for (int j = 0; j < Pairs<T>::N; ++j) top = max_abs(top, v[j]);
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
          const RowScale q = row_scale(top);
          if (!there[u]) continue;
          if (c == 0) a.scale[base + u * RPW + lane / LPR] = q.scale;
          scale_by<T>(v, q.factor);
          store_e4m3<T, false>(static_cast<uint8_t*>(a.out) + at_out, n, a.aligned & AL_OUT, q.finite ? v : Pairs<T>{});
        } else {
          if (!there[u]) continue;
          store_chunk<T, false, WORDS>(static_cast<T*>(a.out) + at_out, n, a.aligned & AL_OUT, packed<T>(v));
        }
      }
    }
  }
  if constexpr (MODE == GRAD) {
    if (!a.partial) return;
#pragma unroll
    for (int j = 0; j < Pairs<T>::N; ++j) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1)
        dw[j] = fadd2(dw[j], make_float2(__shfl_xor_sync(0xffffffffu, dw[j].x, o), __shfl_xor_sync(0xffffffffu, dw[j].y, o)));
      if (lane < LPR) join[warp][c + 2 * j] = dw[j].x, join[warp][c + 2 * j + 1] = dw[j].y;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.C; i += 32 * kNarrowWarps) {
      float s = join[0][i];
#pragma unroll
      for (int g = 1; g < kNarrowWarps; ++g) s += join[g][i];
      a.partial[(int64_t)blockIdx.x * a.C + i] = s;
    }
  }
}

constexpr int kRowWarps = 8;
// Blocks of e4m3 rows that an SM holds: without this bound the weights are fetched before r
// is there, in registers that cost blocks (48828 rows of 2048 bf16 channels 77 us instead of
// 68).  The other modes keep the compiler's own choice (0).
constexpr int e4m3_blocks(int w, int nv, int esz) {
  const int registers = esz == 2 ? (nv == 2 ? (w == 1 ? 64 : 48) : nv == 3 ? (w == 1 ? 80 : 64) : nv == 4 ? 80 : 128)
                                 : (nv == 2 ? (w == 1 ? 48 : 40) : nv == 3 ? (w == 1 ? 64 : 48) : nv == 4 ? 64 : 80);
  const int blocks = 65536 / (registers * 32 * (w == 1 ? kRowWarps : w));
  return blocks > 1 ? blocks : 1;
}

// W warps hold a row in registers, NV chunks of 16 bytes a thread: chunk tid + 32 W i.
// One warp a row: kRowWarps rows a block.
template <typename T, int W, int NV, int MODE, bool WHOLE>
__global__ void __launch_bounds__(W == 1 ? 32 * kRowWarps : 32 * W, MODE == E4M3 ? e4m3_blocks(W, NV, sizeof(T)) : 0) norm_kernel(const Norm a) {
  const int aligned = a.aligned | (WHOLE ? ~0 : 0);
  constexpr int E = 16 / sizeof(T), TPR = 32 * W, ROWS = W == 1 ? kRowWarps : 1;
  __shared__ float2 parts[2][W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = W == 1 ? lane : threadIdx.x;
  int turn = 0;
  // over the threads of a row
  auto row_sum = [&](float2 v) {
    v = MODE == GRAD ? warp_sum2(v) : make_float2(warp_sum1(v.x), 0.f);
    if constexpr (W > 1) {
      if (lane == 0) parts[turn][warp] = v;
      __syncthreads();
      v = parts[turn][0];
#pragma unroll
      for (int i = 1; i < W; ++i) v = fadd2(v, parts[turn][i]);
      turn ^= 1;
    }
    return v;
  };
  auto row_max = [&](float v) {
    v = warp_max1(v);
    if constexpr (W > 1) {
      if (lane == 0) parts[turn][warp].x = v;
      __syncthreads();
      v = parts[turn][0].x;
#pragma unroll
      for (int i = 1; i < W; ++i) v = max_nan(v, parts[turn][i].x);
      turn ^= 1;
    }
    return v;
  };
  const float inv_c = 1.f / (float)a.C;
  Pairs<T> dw[MODE == GRAD ? NV : 1] = {};
  for (int64_t at_row = (int64_t)blockIdx.x * ROWS + (W == 1 ? warp : 0); at_row < a.rows; at_row += (int64_t)gridDim.x * ROWS) {
    const uint32_t row = (uint32_t)at_row, b = row / a.tokens, t = row - b * a.tokens;
    auto at = [&](const int64_t (&s)[2]) { return (int64_t)b * s[0] + (int64_t)t * s[1]; };
    const T* x = static_cast<const T*>(a.x) + at(a.sx);
    const T* res = a.res ? static_cast<const T*>(a.res) + at(a.sres) : nullptr;
    uint4 x_raw[NV], res_raw[NV], dy_raw[MODE == GRAD ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (tid + TPR * i) * E, n = WHOLE ? (a.C - c > 0 ? E : 0) : a.C - c;
      x_raw[i] = make_uint4(0, 0, 0, 0);
      if (n > 0) x_raw[i] = load_chunk<T, WHOLE>(x + c, n, aligned & AL_X);
    }
    if (res) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = WHOLE ? (a.C - c > 0 ? E : 0) : a.C - c;
        res_raw[i] = make_uint4(0, 0, 0, 0);
        if (n > 0) res_raw[i] = load_chunk<T, WHOLE>(res + c, n, aligned & AL_RES);
      }
    }
    if constexpr (MODE == GRAD) {
      const T* dy = static_cast<const T*>(a.dy) + at(a.sdy);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = WHOLE ? (a.C - c > 0 ? E : 0) : a.C - c;
        dy_raw[i] = make_uint4(0, 0, 0, 0);
        if (n > 0) dy_raw[i] = load_chunk<T, WHOLE>(dy + c, n, aligned & AL_DY);
      }
      float2 square = make_float2(0.f, 0.f), dot = square;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = WHOLE ? (a.C - c > 0 ? E : 0) : a.C - c;
        const Pairs<T> v = pairs<T>(x_raw[i]);
        Pairs<T> g = pairs<T>(dy_raw[i]);
        times_weight<T, WHOLE>(g, a.w, c, n, aligned & AL_W);
        add_products<T>(square, v, v);
        add_products<T>(dot, g, v);
      }
      const float2 sums = row_sum(make_float2(square.x + square.y, dot.x + dot.y));
      const float r = rsqrtf(fmaf(sums.x, inv_c, a.eps)), k = r * r * (sums.y * inv_c);
      T* out = static_cast<T*>(a.out) + at(a.sout);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = WHOLE ? (a.C - c > 0 ? E : 0) : a.C - c;
        if (n <= 0) continue;
        const Pairs<T> v = pairs<T>(x_raw[i]), g = pairs<T>(dy_raw[i]);
        Pairs<T> d = g;
        times_weight<T, WHOLE>(d, a.w, c, n, aligned & AL_W);
        norm_gradient<T>(g, d, v, r, k, dw[i]);
        if (res) add_to<T>(d, pairs<T>(res_raw[i]));
        store_chunk<T, WHOLE>(out + c, n, aligned & AL_OUT, packed<T>(d));
      }
    } else {
      Pairs<T> v[NV];
      float2 square = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = WHOLE ? (a.C - c > 0 ? E : 0) : a.C - c;
        v[i] = pairs<T>(x_raw[i]);
        if (res) {
          add_to<T>(v[i], pairs<T>(res_raw[i]));
          const uint4 sum = packed<T>(v[i]);
          v[i] = pairs<T>(sum);  // the norm is of the sum as it is kept
          if (a.total && n > 0) store_chunk<T, WHOLE>(static_cast<T*>(a.total) + at(a.stotal) + c, n, aligned & AL_TOTAL, sum);
        }
        add_products<T>(square, v[i], v[i]);
      }
      const float r = rsqrtf(fmaf(row_sum(make_float2(square.x + square.y, 0.f)).x, inv_c, a.eps));
      float factor = 1.f, top = 0.f;
      bool finite = true;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = WHOLE ? (a.C - c > 0 ? E : 0) : a.C - c;
        scale_by<T>(v[i], r);
        times_weight<T, WHOLE>(v[i], a.w, c, n, aligned & AL_W);
        if constexpr (MODE == E4M3)
#pragma unroll
          for (int j = 0; j < Pairs<T>::N; ++j) top = max_abs(top, v[i][j]);
      }
      if constexpr (MODE == E4M3) {
        const RowScale q = row_scale(row_max(top));
        factor = q.factor, finite = q.finite;
        if (tid == 0) a.scale[row] = q.scale;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = WHOLE ? (a.C - c > 0 ? E : 0) : a.C - c;
        if (n <= 0) continue;
        if constexpr (MODE == E4M3) scale_by<T>(v[i], factor);
        if constexpr (MODE == E4M3) store_e4m3<T, WHOLE>(static_cast<uint8_t*>(a.out) + at(a.sout) + c, n, aligned & AL_OUT, finite ? v[i] : Pairs<T>{});
        else store_chunk<T, WHOLE>(static_cast<T*>(a.out) + at(a.sout) + c, n, aligned & AL_OUT, packed<T>(v[i]));
      }
    }
  }
  if constexpr (MODE == GRAD) {
    if (!a.partial) return;
    float* partial = a.partial + (int64_t)blockIdx.x * a.C;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int c = (tid + TPR * i) * E + j;
        if (c < a.C) partial[c] = j & 1 ? dw[i][j / 2].y : dw[i][j / 2].x;
      }
    }
  }
}

// Rows that one strand of a weight sum adds up one after the other, at most.
constexpr int64_t kSerialRows = 256;
constexpr int kNormSms = 152;

inline int chunks_of(int C, int esz) { return (C * esz + 15) / 16; }
// How rows of so many chunks are held: narrow (lanes a row), a ring (warps a row, chunks
// a thread, rows a block), or, fp32 rows past 8192 channels, the registers of a block.
struct Shape {
  int lanes, rw, nv, rows;
};
// WHOLE: every tensor lies in rows of whole 16-byte vectors, and there is a weight;
// ALIGNED: rows that begin at such vectors; ODD: any.
enum Rows { WHOLE_ROWS, ALIGNED_ROWS, ODD_ROWS };
// Odd rows of more than 20 chunks fare better with shifted windows (411206 rows of 255
// bf16 channels 268 us, 457 element by element; of 130, 17 chunks, 513 and 475, and
// 277 by words).
inline Shape shape_of(int chunks, Rows kind) {
  for (const int lanes : {1, 4, 8, 16, 32})
    if (chunks <= lanes && (kind != ODD_ROWS || chunks <= 20)) return {lanes, 0, 0, kNarrowWarps * 32 / lanes};
  for (const Shape w : {Shape{0, 1, 1, 4}, {0, 1, 2, 4}, {0, 2, 2, 4}, {0, 2, 3, 4}, {0, 4, 2, 2}, {0, 4, 4, 2}, {0, 8, 4, 1}, {0, 16, 4, 1}})
    if (chunks <= 32 * w.rw * w.nv) return w;
  return {0, 0, 0, 1};
}
// Blocks: what the card holds at once; of the gradient enough that no strand is longer than kSerialRows.
inline int64_t blocks_of(const dit_rms_norm_args& a, bool backward, Rows kind) {
  const Shape w = shape_of(chunks_of(a.channels, a.dtype == DIT_DTYPE_F32 ? 4 : 2), kind);
  const int64_t rows = a.batch * a.tokens, at_once = w.rows * (w.lanes ? kNarrowBatch : 1), most = (rows + at_once - 1) / at_once;
  int64_t n = kNormSms * (w.lanes ? (backward ? 8 : 32) : w.rw ? ring_blocks(w.rw, w.nv, w.rows, 1 + (backward ? 1 : 0) + (a.residual ? 1 : 0), backward && kind != WHOLE_ROWS) : backward ? 2 : 64);
  // the forward's last blocks wait less for each other when there are more of them
  // (204800 odd rows of 512 172 us, 205 with one for each place)
  if (!backward && w.rw) n *= 4;
  const int64_t least = (rows + w.rows * kSerialRows - 1) / (w.rows * kSerialRows);
  if (backward && n < least) n = least;
  return n < most ? n : most;
}

template <typename T, int RW, int NV, int ROWS, int MODE, bool RES, bool WHOLE>
cudaError_t launch_ring(const Norm& p, int64_t blocks, cudaStream_t s) {
  return launch_kernel(norm_ring_kernel<T, RW, NV, ROWS, MODE, RES, WHOLE>, dim3((unsigned)blocks), dim3(32 * RW * ROWS),
                       Ring<RW, NV, ROWS, MODE, RES, WHOLE>::SMEM + ROWS * 2 * RW * sizeof(float2), s, 1, false, p);
}
template <typename T, int RW, int NV, int ROWS, int MODE>
cudaError_t ring(const Norm& p, bool whole, int64_t blocks, cudaStream_t s) {
  if constexpr (MODE == GRAD)
    if (whole) return p.res ? launch_ring<T, RW, NV, ROWS, MODE, true, true>(p, blocks, s) : launch_ring<T, RW, NV, ROWS, MODE, false, true>(p, blocks, s);
  return p.res ? launch_ring<T, RW, NV, ROWS, MODE, true, false>(p, blocks, s) : launch_ring<T, RW, NV, ROWS, MODE, false, false>(p, blocks, s);
}
template <typename T, int LPR, int MODE>
cudaError_t narrow(const Norm& p, int64_t blocks, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (p.words) return launch_kernel(norm_narrow_kernel<T, LPR, MODE, true>, dim3((unsigned)blocks), dim3(32 * kNarrowWarps), 0, s, 1, false, p);
  return launch_kernel(norm_narrow_kernel<T, LPR, MODE, false>, dim3((unsigned)blocks), dim3(32 * kNarrowWarps), 0, s, 1, false, p);
}
template <typename T, int W, int NV, int MODE, bool WHOLE>
cudaError_t launch_rows(const Norm& p, int64_t blocks, cudaStream_t s) {
  if (W == 1) blocks = (p.rows + kRowWarps - 1) / kRowWarps;
  return launch_kernel(norm_kernel<T, W, NV, MODE, WHOLE>, dim3((unsigned)blocks), dim3(W == 1 ? 32 * kRowWarps : 32 * W), 0, s, 1, false, p);
}
inline Rows rows_kind(const Norm& p, int E) {
  const int need = AL_X | AL_OUT | (p.res ? AL_RES : 0) | (p.total ? AL_TOTAL : 0) | (p.dy ? AL_DY : 0);
  if ((p.aligned & need) != need) return ODD_ROWS;
  return (p.aligned & AL_W) && p.C % E == 0 && p.w ? WHOLE_ROWS : ALIGNED_ROWS;
}
// Whole rows of a forward call are held in registers, without copies (the video pair
// 112 us, 129 us through the ring; e4m3 54 and 75); all others go through the ring.
template <typename T, int MODE>
cudaError_t by_width(const Norm& p, int64_t blocks, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  const int chunks = chunks_of(p.C, sizeof(T));
  const Rows kind = rows_kind(p, E);
  const bool whole = kind == WHOLE_ROWS;
  if (chunks <= 1) return narrow<T, 1, MODE>(p, blocks, s);
  if (chunks <= 4) return narrow<T, 4, MODE>(p, blocks, s);
  if (chunks <= 8) return narrow<T, 8, MODE>(p, blocks, s);
  if (chunks <= 16) return narrow<T, 16, MODE>(p, blocks, s);
  if (chunks <= (kind == ODD_ROWS ? 20 : 32)) return narrow<T, 32, MODE>(p, blocks, s);
  if (chunks <= 32) return ring<T, 1, 1, 4, MODE>(p, false, blocks, s);
  if constexpr (MODE != GRAD) {
    if (whole) {
      // warps a row: 51200 rows of 2048 in e4m3 109 us on four, 136 on one; 68266 of 1536
      // with a residual 122 on one, 126 on two, without one 79 and 66.  10^8 bf16 values with a
      // residual on one and on two: 1280 channels 116 and 121, 1152 118 and 118, 1032 126 and
      // 120, into e4m3 114 and 108, 120 and 107, 128 and 112 (1536 106 both); fp32 768 227 and 238
      if (chunks <= 64) return launch_rows<T, 1, 2, MODE, true>(p, blocks, s);
      if (chunks <= 96) return launch_rows<T, 1, 3, MODE, true>(p, blocks, s);
      if (chunks > 128 && chunks <= 192 && p.res) return launch_rows<T, 1, 6, MODE, true>(p, blocks, s);
      blocks = p.rows < kNormSms * 64u ? p.rows : kNormSms * 64u;
      if (chunks <= 128) return launch_rows<T, 2, 2, MODE, true>(p, blocks, s);
      if (chunks <= 192) return launch_rows<T, 2, 3, MODE, true>(p, blocks, s);
      if (chunks <= 256) return launch_rows<T, 4, 2, MODE, true>(p, blocks, s);
      if (chunks <= 512) return launch_rows<T, 4, 4, MODE, true>(p, blocks, s);
      if (chunks <= 1024) return launch_rows<T, 8, 4, MODE, true>(p, blocks, s);
      if (chunks <= 2048) return launch_rows<T, 16, 4, MODE, true>(p, blocks, s);
      if constexpr (E == 4) return launch_rows<T, 32, 4, MODE, true>(p, blocks, s);
    }
  }
  if (chunks <= 64) return ring<T, 1, 2, 4, MODE>(p, whole, blocks, s);
  if (chunks <= 128) return ring<T, 2, 2, 4, MODE>(p, whole, blocks, s);
  if (chunks <= 192) return ring<T, 2, 3, 4, MODE>(p, whole, blocks, s);
  if (chunks <= 256) return ring<T, 4, 2, 2, MODE>(p, whole, blocks, s);
  if (chunks <= 512) return ring<T, 4, 4, 2, MODE>(p, whole, blocks, s);
  if (chunks <= 1024) return ring<T, 8, 4, 1, MODE>(p, whole, blocks, s);
  if (chunks <= 2048) return ring<T, 16, 4, 1, MODE>(p, whole, blocks, s);
  if constexpr (E == 4) return launch_rows<T, 32, 4, MODE, false>(p, blocks, s);
  return cudaErrorInvalidValue;
}

// All kernels of one activation type; an instance in a source file of its own.
template <typename T>
cudaError_t by_mode(const Norm& p, int mode, int64_t blocks, cudaStream_t s) {
  return mode == GRAD ? by_width<T, GRAD>(p, blocks, s) : mode == E4M3 ? by_width<T, E4M3>(p, blocks, s) : by_width<T, SAME>(p, blocks, s);
}
extern template cudaError_t by_mode<float>(const Norm&, int, int64_t, cudaStream_t);
extern template cudaError_t by_mode<__nv_bfloat16>(const Norm&, int, int64_t, cudaStream_t);
extern template cudaError_t by_mode<__half>(const Norm&, int, int64_t, cudaStream_t);

}  // namespace norm

}  // namespace dit
