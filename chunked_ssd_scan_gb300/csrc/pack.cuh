// Vectors of up to 16 bytes of an I/O tensor as fp32 pairs.
#pragma once

#include <string.h>

#include "common.cuh"

namespace ssd {

template <int kBytes>
struct RawOf;
template <>
struct RawOf<16> { using type = uint4; };
template <>
struct RawOf<8> { using type = uint2; };
template <>
struct RawOf<4> { using type = uint32_t; };
template <>
struct RawOf<2> { using type = uint16_t; };

// V neighbouring values as one load or store of up to 16 bytes (Raw, as they wait for their turn), in P
// pairs (V = 1: the second is 0).
template <typename T, int V>
struct Pack {
  static constexpr int P = (V + 1) / 2;
  using Raw = typename RawOf<V * (int)sizeof(T)>::type;
  static __device__ __forceinline__ Raw raw(const T* p) { return __ldg(reinterpret_cast<const Raw*>(p)); }
  static __device__ __forceinline__ Raw none() {
    Raw r;
    memset(&r, 0, sizeof(r));
    return r;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float2 (&f)[P]) {
    if constexpr (sizeof(T) == 2) {
      if constexpr (V == 1) {
        f[0] = make_float2(__uint_as_float((uint32_t)r << 16), 0.f);
      } else {
        uint32_t u[P];
        memcpy(u, &r, sizeof(r));
#pragma unroll
        for (int k = 0; k < P; ++k)
          f[k] = make_float2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u));
      }
    } else {
      float v[2 * P] = {};
      memcpy(v, &r, sizeof(r));
#pragma unroll
      for (int k = 0; k < P; ++k) f[k] = make_float2(v[2 * k], v[2 * k + 1]);
    }
  }
  static __device__ __forceinline__ void store(T* p, const float2 (&f)[P]) {
    if constexpr (V == 1) {
      st_from_f32(p, f[0].x);
    } else if constexpr (sizeof(T) == 2) {
      uint32_t u[P];
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[k].x, f[k].y);
        u[k] = *reinterpret_cast<const uint32_t*>(&b);
      }
      if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(u);
      else if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(u);
      else *reinterpret_cast<uint32_t*>(p) = u[0];
    } else {
      if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
      else *reinterpret_cast<float2*>(p) = f[0];
    }
  }
  static __device__ __forceinline__ void param(const float* p, int64_t at, float none, float2 (&f)[P]) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      f[k].x = p ? __ldg(p + at + 2 * k) : none;
      f[k].y = V == 1 ? 0.f : p ? __ldg(p + at + 2 * k + 1) : none;
    }
  }
  static __device__ __forceinline__ void zero(float2 (&f)[P]) {
#pragma unroll
    for (int k = 0; k < P; ++k) f[k] = make_float2(0.f, 0.f);
  }
};

}  // namespace ssd
