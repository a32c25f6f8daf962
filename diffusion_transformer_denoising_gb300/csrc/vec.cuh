// Typed 8-element and single-element accesses of the operators on fp32, bf16
// and fp16 activations: values are fp32 in registers, rounded once (to
// nearest even) when they are stored.  And the exact sum of two floats.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace dit {

// a + b = high + low exactly (Knuth).
DIT_DEV float two_sum(float a, float b, float& low) {
  const float h = a + b, t = h - a;
  low = (a - (h - t)) + (b - t);
  return h;
}
// A sum taken one term after the other that loses nothing: high and low part.
struct LongSum {
  float h = 0.f, l = 0.f;
  DIT_DEV void add(float v) {
    float t;
    h = two_sum(h, v, t);
    l += t;
  }
  DIT_DEV float value() const { return isfinite(h) ? h + l : h; }
};

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

// N elements of T as they lie in memory: 16-byte words, one word of 8 or 4
// bytes, or a single element.  A pointer to them is aligned to the word.
template <typename T, int N>
struct Raw {
  static constexpr int kBytes = N * sizeof(T);
  static constexpr int kWords = kBytes / 4 > 0 ? kBytes / 4 : 1;
  uint32_t w[kWords];
};

template <typename T, int N>
DIT_DEV Raw<T, N> load_raw(const T* p) {
  Raw<T, N> r;
  constexpr int B = Raw<T, N>::kBytes;
  if constexpr (B >= 16) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
  } else if constexpr (B == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  } else if constexpr (B == 4) {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  }
  return r;
}
template <typename T, int N>
DIT_DEV Raw<T, N> zero_raw() {
  Raw<T, N> r;
#pragma unroll
  for (int i = 0; i < Raw<T, N>::kWords; ++i) r.w[i] = 0;
  return r;
}
template <typename T, int N>
DIT_DEV void unpack(const Raw<T, N>& r, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < Raw<T, N>::kWords; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = __uint_as_float(r.w[i]);
    } else {
      const float2 t = unpack2<T>(r.w[i]);
      f[2 * i] = t.x;
      if constexpr (N > 1) f[2 * i + 1] = t.y;
    }
  }
}
template <typename T, int N, bool STREAM = false>
DIT_DEV void store_f32(T* p, const float (&f)[N]) {
  constexpr int B = Raw<T, N>::kBytes;
  if constexpr (N == 1) {
    *p = from_f32<T>(f[0]);
  } else {
    uint32_t w[Raw<T, N>::kWords];
#pragma unroll
    for (int i = 0; i < Raw<T, N>::kWords; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
      else w[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
    }
    if constexpr (B >= 16) {
#pragma unroll
      for (int i = 0; i < B / 16; ++i) {
        const uint4 v = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        if constexpr (STREAM) __stcs(reinterpret_cast<uint4*>(p) + i, v);
        else reinterpret_cast<uint4*>(p)[i] = v;
      }
    } else if constexpr (B == 8) {
      if constexpr (STREAM) __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
      else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    }
  }
}
// Evict-first: results that nothing of this call reads again.
template <typename T, int N>
DIT_DEV void store_f32_stream(T* p, const float (&f)[N]) {
  store_f32<T, N, true>(p, f);
}

}  // namespace dit
