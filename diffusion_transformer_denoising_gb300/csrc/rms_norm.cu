// RMS norm over channels with the residual's addition in front of it, into the
// activations' type or into e4m3 with a scale for each row, and its gradient.
//
// Mathematics.  v = x + residual rounded to the type, r = (mean v^2 + eps)^-1/2,
// y = v r w.  e4m3: scale = max |y| / 448, y / scale rounded to nearest even.
// Gradient: g = dy w, dx = dtotal + r (g - v r^2 mean(g v)), dw = sum dy v r: the two
// row sums (v^2 and g v) are taken together.
//
// What bounds it: HBM.  Every row is read once, held in registers and written
// once: by a warp up to 2048 channels of 16 bits (1024 of 32), by a block beyond.
#include <math.h>

#include "column_sums.cuh"
#include "launch.cuh"
#include "operators.h"
#include "vec.cuh"

namespace dit {

namespace {

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
};

DIT_DEV float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// E elements from p on, of which n are there (0 behind them).
template <typename T, int E>
DIT_DEV Raw<T, E> load_some(const T* p, int n, bool aligned) {
  if (n >= E && aligned) return load_raw<T, E>(p);
  Raw<T, E> r = zero_raw<T, E>();
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < n) r.w[j] = __float_as_uint(to_f32(p[j]));
  } else {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < n) r.w[j / 2] |= (uint32_t)q[j] << (16 * (j & 1));
  }
  return r;
}
template <typename T, int E>
DIT_DEV void store_some(T* p, int n, bool aligned, const float (&v)[E]) {
  if (n >= E && aligned) {
    store_f32<T, E>(p, v);
    return;
  }
#pragma unroll
  for (int j = 0; j < E; ++j)
    if (j < n) p[j] = from_f32<T>(v[j]);
}
template <int E>
DIT_DEV void store_e4m3(uint8_t* p, int n, bool aligned, const float (&v)[E]) {
  uint32_t w[E / 4];
#pragma unroll
  for (int j = 0; j < E / 4; ++j) w[j] = pack_e4m3x4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  if (n >= E && aligned) {
    if constexpr (E == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
    return;
  }
#pragma unroll
  for (int j = 0; j < E; ++j)
    if (j < n) p[j] = (uint8_t)(w[j / 4] >> (8 * (j & 3)));
}
template <int E>
DIT_DEV void load_weight(const float* w, int c, int n, bool aligned, float (&v)[E]) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = 1.f;
  } else if (n >= E && aligned) {
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(w + c + j));
      v[j] = t.x, v[j + 1] = t.y, v[j + 2] = t.z, v[j + 3] = t.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = j < n ? __ldg(w + c + j) : 0.f;
  }
}

// W warps hold a row, NV chunks of 16 bytes a thread: chunk tid + 32 W i.  One
// warp a row: eight rows a block.
template <typename T, int W, int NV, int MODE>
__global__ void __launch_bounds__(W == 1 ? 256 : 32 * W) norm_kernel(const Norm a) {
  constexpr int E = 16 / sizeof(T), TPR = 32 * W, GROUPS = W == 1 ? 8 : 1;
  __shared__ float2 parts[2][W];
  __shared__ float columns[MODE == GRAD && W == 1 ? GROUPS * 32 * (E + 1) : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = W == 1 ? lane : threadIdx.x;
  int turn = 0;
  // sums (or, of e4m3, maxima) over the threads of a row
  auto row_sum = [&](float2 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      if (MODE == GRAD) v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (W > 1) {
      if (lane == 0) parts[turn][warp] = v;
      __syncthreads();
      v = parts[turn][0];
#pragma unroll
      for (int i = 1; i < W; ++i) v.x += parts[turn][i].x, v.y += parts[turn][i].y;
      turn ^= 1;
    }
    return v;
  };
  auto row_max = [&](float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
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
  float dw[MODE == GRAD ? NV : 1][E] = {};
  for (uint32_t row = blockIdx.x * GROUPS + (W == 1 ? warp : 0); row < a.rows; row += gridDim.x * GROUPS) {
    const uint32_t b = row / a.tokens, t = row - b * a.tokens;
    auto at = [&](const int64_t (&s)[2]) { return (int64_t)b * s[0] + (int64_t)t * s[1]; };
    const T* x = static_cast<const T*>(a.x) + at(a.sx);
    const T* res = static_cast<const T*>(a.res) + (a.res ? at(a.sres) : 0);
    Raw<T, E> v[NV], q[NV], d[MODE == GRAD ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (tid + TPR * i) * E, n = a.C - c;
      v[i] = zero_raw<T, E>();
      if (n > 0) v[i] = load_some<T, E>(x + c, n, a.aligned & AL_X);
    }
    if (a.res) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = a.C - c;
        q[i] = zero_raw<T, E>();
        if (n > 0) q[i] = load_some<T, E>(res + c, n, a.aligned & AL_RES);
      }
    }
    if constexpr (MODE == GRAD) {
      const T* dy = static_cast<const T*>(a.dy) + at(a.sdy);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = a.C - c;
        d[i] = zero_raw<T, E>();
        if (n > 0) d[i] = load_some<T, E>(dy + c, n, a.aligned & AL_DY);
      }
    }
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (tid + TPR * i) * E, n = a.C - c;
      float f[E];
      unpack<T, E>(v[i], f);
      if constexpr (MODE != GRAD) {
        if (a.res) {
          float g[E];
          unpack<T, E>(q[i], g);
#pragma unroll
          for (int j = 0; j < E; ++j) f[j] = to_f32(from_f32<T>(f[j] + g[j]));
          if (a.total && n > 0) store_some<T, E>(static_cast<T*>(a.total) + at(a.stotal) + c, n, a.aligned & AL_TOTAL, f);
          // what the norm is of: the sum as it is kept
#pragma unroll
          for (int j = 0; j < Raw<T, E>::kWords; ++j) {
            if constexpr (sizeof(T) == 4) v[i].w[j] = __float_as_uint(f[j]);
            else v[i].w[j] = pack2<T>(f[2 * j], f[2 * j + 1]);
          }
        }
#pragma unroll
        for (int j = 0; j < E; ++j) sum.x = fmaf(f[j], f[j], sum.x);
      } else {
        float g[E], w[E];
        unpack<T, E>(d[i], g);
        load_weight<E>(a.w, c, n, a.aligned & AL_W, w);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          sum.x = fmaf(f[j], f[j], sum.x);
          sum.y = fmaf(g[j] * w[j], f[j], sum.y);
        }
      }
    }
    sum = row_sum(sum);
    const float r = rsqrtf(fmaf(sum.x, inv_c, a.eps));
    if constexpr (MODE == SAME) {
      T* out = static_cast<T*>(a.out) + at(a.sout);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = a.C - c;
        if (n <= 0) continue;
        float f[E], w[E];
        unpack<T, E>(v[i], f);
        load_weight<E>(a.w, c, n, a.aligned & AL_W, w);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] *= r * w[j];
        store_some<T, E>(out + c, n, a.aligned & AL_OUT, f);
      }
    } else if constexpr (MODE == E4M3) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = a.C - c;
        if (n <= 0) continue;
        float f[E], w[E];
        unpack<T, E>(v[i], f);
        load_weight<E>(a.w, c, n, a.aligned & AL_W, w);
#pragma unroll
        for (int j = 0; j < E; ++j) top = max_nan(top, fabsf(f[j] * (r * w[j])));
      }
      top = row_max(top);
      const bool finite = top <= 3.402823466e38f;
      // below 448 x 2^-126 the scale stays a normal number, so that its reciprocal is finite
      const float scale = !finite ? __int_as_float(0x7fffffff) : top > 0.f ? fmaxf(top / kE4M3Max, 1.17549435e-38f) : 1.f;
      const float k = finite ? r / scale : 0.f;
      uint8_t* out = static_cast<uint8_t*>(a.out) + at(a.sout);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = a.C - c;
        if (n <= 0) continue;
        float f[E], w[E];
        unpack<T, E>(v[i], f);
        load_weight<E>(a.w, c, n, a.aligned & AL_W, w);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = finite ? f[j] * (k * w[j]) : 0.f;
        store_e4m3<E>(out + c, n, a.aligned & AL_OUT, f);
      }
      if (tid == 0) a.scale[row] = scale;
    } else {
      const float k = r * r * (sum.y * inv_c);
      T* out = static_cast<T*>(a.out) + at(a.sout);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + TPR * i) * E, n = a.C - c;
        if (n <= 0) continue;
        float f[E], g[E], w[E], o[E];
        unpack<T, E>(v[i], f);
        unpack<T, E>(d[i], g);
        load_weight<E>(a.w, c, n, a.aligned & AL_W, w);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          dw[i][j] = fmaf(g[j], f[j] * r, dw[i][j]);
          o[j] = r * fmaf(-k, f[j], g[j] * w[j]);
        }
        if (a.res) {
          unpack<T, E>(q[i], f);
#pragma unroll
          for (int j = 0; j < E; ++j) o[j] += f[j];
        }
        store_some<T, E>(out + c, n, a.aligned & AL_OUT, o);
      }
    }
  }
  if constexpr (MODE == GRAD) {
    if (!a.partial) return;
    float* partial = a.partial + (int64_t)blockIdx.x * a.C;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (W == 1) {
        // the eight warps' sums of 32 E columns
#pragma unroll
        for (int j = 0; j < E; ++j) columns[(warp * 32 + lane) * (E + 1) + j] = dw[i][j];
        __syncthreads();
        for (int k = threadIdx.x; k < 32 * E; k += 256) {
          float s = 0.f;
#pragma unroll
          for (int g = 0; g < GROUPS; ++g) s += columns[(g * 32 + k / E) * (E + 1) + k % E];
          const int c = 32 * E * i + k;
          if (c < a.C) partial[c] = s;
        }
        __syncthreads();
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const int c = (tid + TPR * i) * E + j;
          if (c < a.C) partial[c] = dw[i][j];
        }
      }
    }
  }
}

// Rows that one strand of a weight sum adds up one after the other, at most.
constexpr int64_t kSerialRows = 256;
constexpr int kNormSms = 152;

int warps_per_row(const dit_rms_norm_args& a) {
  const int chunk = a.dtype == DIT_DTYPE_F32 ? 4 : 8;
  const int chunks = (a.channels + chunk - 1) / chunk;
  return chunks <= 32 * 8 ? 1 : chunks <= 128 * 4 ? 4 : chunks <= 256 * 4 ? 8 : chunks <= 512 * 4 ? 16 : 32;
}
// Blocks of the gradient: enough to fill the card and that no strand is longer than kSerialRows.
int64_t grad_blocks(const dit_rms_norm_args& a) {
  const int w = warps_per_row(a), groups = w == 1 ? 8 : 1;
  const int64_t rows = a.batch * a.tokens;
  int64_t n = kNormSms * (w <= 4 ? 2 : 1);
  const int64_t least = (rows + groups * kSerialRows - 1) / (groups * kSerialRows), most = (rows + groups - 1) / groups;
  n = n < least ? least : n;
  return n < most ? n : most;
}

template <typename T, int W, int NV, int MODE>
cudaError_t launch(const Norm& p, int64_t blocks, cudaStream_t s) {
  return launch_kernel(norm_kernel<T, W, NV, MODE>, dim3((unsigned)blocks), dim3(W == 1 ? 256 : 32 * W), 0, s, 1, false, p);
}
template <typename T, int MODE>
cudaError_t by_width(const Norm& p, int64_t blocks, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  const int chunks = (p.C + E - 1) / E;
  if (chunks <= 32) return launch<T, 1, 1, MODE>(p, blocks, s);
  if (chunks <= 64) return launch<T, 1, 2, MODE>(p, blocks, s);
  if (chunks <= 128) return launch<T, 1, 4, MODE>(p, blocks, s);
  if (chunks <= 192) return launch<T, 1, 6, MODE>(p, blocks, s);
  if (chunks <= 256) return launch<T, 1, 8, MODE>(p, blocks, s);
  if (chunks <= 512) return launch<T, 4, 4, MODE>(p, blocks, s);
  if (chunks <= 1024) return launch<T, 8, 4, MODE>(p, blocks, s);
  if (chunks <= 2048) return launch<T, 16, 4, MODE>(p, blocks, s);
  if constexpr (E == 4) return launch<T, 32, 4, MODE>(p, blocks, s);
  return cudaErrorInvalidValue;
}
template <int MODE>
cudaError_t by_type(int dtype, const Norm& p, int64_t blocks, cudaStream_t s) {
  if (dtype == DIT_DTYPE_F32) return by_width<float, MODE>(p, blocks, s);
  if (dtype == DIT_DTYPE_BF16) return by_width<__nv_bfloat16, MODE>(p, blocks, s);
  return by_width<__half, MODE>(p, blocks, s);
}

}  // namespace

int64_t rms_norm_workspace(const dit_rms_norm_args& a) {
  return a.dweight && a.batch * a.tokens ? grad_blocks(a) * a.channels * (int64_t)sizeof(float) : 0;
}

cudaError_t rms_norm_run(const dit_rms_norm_args& a, bool backward, float* workspace, cudaStream_t s) {
  const int64_t rows = a.batch * a.tokens;
  if (rows == 0) return a.dweight ? cudaMemsetAsync(a.dweight, 0, (size_t)a.channels * 4, s) : cudaSuccess;
  Norm p{};
  p.x = a.x, p.res = a.residual, p.dy = a.dy, p.total = a.total, p.out = a.out;
  const int esz = a.dtype == DIT_DTYPE_F32 ? 4 : 2;
  const int out_bytes = a.out_dtype == DIT_DTYPE_E4M3 ? 16 / esz : 16, out_esz = a.out_dtype == DIT_DTYPE_E4M3 ? 1 : esz;
  for (int i = 0; i < 2; ++i) {
    p.sx[i] = a.x_stride[i], p.sres[i] = a.residual_stride[i], p.stotal[i] = a.total_stride[i];
    p.sdy[i] = a.dy_stride[i], p.sout[i] = a.out_stride[i];
  }
  auto aligned = [&](const void* q, const int64_t (&st)[2], int e, int bytes) {
    return (((uintptr_t)q | (uintptr_t)(st[0] * e) | (uintptr_t)(st[1] * e)) & (bytes - 1)) == 0;
  };
  p.aligned = (aligned(p.x, p.sx, esz, 16) ? AL_X : 0) | (aligned(p.res, p.sres, esz, 16) ? AL_RES : 0) |
              (aligned(p.total, p.stotal, esz, 16) ? AL_TOTAL : 0) | (aligned(p.dy, p.sdy, esz, 16) ? AL_DY : 0) |
              (aligned(p.out, p.sout, out_esz, out_bytes) ? AL_OUT : 0) | (((uintptr_t)a.weight & 15) == 0 ? AL_W : 0);
  p.scale = a.scale, p.w = a.weight;
  p.rows = (uint32_t)rows, p.tokens = (uint32_t)a.tokens;
  p.C = a.channels, p.eps = a.eps;
  if (!backward) {
    const int w = warps_per_row(a), groups = w == 1 ? 8 : 1;
    const int64_t most = (rows + groups - 1) / groups, fill = kNormSms * 64ll;
    const int64_t blocks = most < fill ? most : fill;
    return a.out_dtype == DIT_DTYPE_E4M3 ? by_type<E4M3>(a.dtype, p, blocks, s) : by_type<SAME>(a.dtype, p, blocks, s);
  }
  const int64_t blocks = grad_blocks(a);
  p.partial = a.dweight ? workspace : nullptr;
  const cudaError_t e = by_type<GRAD>(a.dtype, p, blocks, s);
  if (e != cudaSuccess || !a.dweight) return e;
  return column_sums(ColumnSums{workspace, blocks, a.channels, a.channels, 0, {a.dweight, nullptr}}, s);
}

}  // namespace dit
