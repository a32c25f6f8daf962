// Typed 8-element and single-element accesses of the operators on fp32, bf16
// and fp16 activations: values are fp32 in registers, rounded once (to
// nearest even) when they are stored.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace dit {

DIT_DEV float to_f32(float v) { return v; }
DIT_DEV float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
DIT_DEV float to_f32(__half v) { return __half2float(v); }
template <typename T>
DIT_DEV T from_f32(float v);
template <>
DIT_DEV float from_f32<float>(float v) { return v; }
template <>
DIT_DEV __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
DIT_DEV __half from_f32<__half>(float v) { return __float2half_rn(v); }

template <typename T>
DIT_DEV float2 unpack2(uint32_t u);
template <>
DIT_DEV float2 unpack2<__nv_bfloat16>(uint32_t u) { return make_float2(bf16_lo(u), bf16_hi(u)); }
template <>
DIT_DEV float2 unpack2<__half>(uint32_t u) { return __half22float2(*reinterpret_cast<__half2*>(&u)); }
template <typename T>
DIT_DEV uint32_t pack2(float lo, float hi);
template <>
DIT_DEV uint32_t pack2<__nv_bfloat16>(float lo, float hi) { return pack_bf16x2(lo, hi); }
template <>
DIT_DEV uint32_t pack2<__half>(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// N elements of T as raw 16-byte words (N * sizeof(T) a multiple of 16), and
// N = 1 as the element itself.
template <typename T, int N>
struct Raw {
  uint4 v[N * sizeof(T) / 16];
};
template <typename T>
struct Raw<T, 1> {
  T v;
};

template <typename T, int N>
DIT_DEV Raw<T, N> load_raw(const T* p) {
  Raw<T, N> r;
  if constexpr (N == 1) {
    r.v = *p;
  } else {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  return r;
}
template <typename T, int N>
DIT_DEV Raw<T, N> zero_raw() {
  Raw<T, N> r;
  if constexpr (N == 1) {
    r.v = from_f32<T>(0.f);
  } else {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) r.v[i] = make_uint4(0, 0, 0, 0);
  }
  return r;
}
template <typename T, int N>
DIT_DEV void unpack(const Raw<T, N>& r, float (&f)[N]) {
  if constexpr (N == 1) {
    f[0] = to_f32(r.v);
  } else {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) {
      const uint32_t w[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          f[4 * i + j] = __uint_as_float(w[j]);
        } else {
          const float2 t = unpack2<T>(w[j]);
          f[8 * i + 2 * j] = t.x;
          f[8 * i + 2 * j + 1] = t.y;
        }
      }
    }
  }
}
template <typename T, int N>
DIT_DEV void store_f32(T* p, const float (&f)[N]) {
  if constexpr (N == 1) {
    *p = from_f32<T>(f[0]);
  } else {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) {
      uint4 v;
      if constexpr (sizeof(T) == 4) {
        v = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                       __float_as_uint(f[4 * i + 3]));
      } else {
        v = make_uint4(pack2<T>(f[8 * i], f[8 * i + 1]), pack2<T>(f[8 * i + 2], f[8 * i + 3]),
                       pack2<T>(f[8 * i + 4], f[8 * i + 5]), pack2<T>(f[8 * i + 6], f[8 * i + 7]));
      }
      reinterpret_cast<uint4*>(p)[i] = v;
    }
  }
}

}  // namespace dit
