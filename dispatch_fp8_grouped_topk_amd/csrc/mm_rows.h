// Rows of values as the elementwise kernels take them: eight consecutive columns a lane (16 bytes of BF16, 32 of
// float32), so that a group of 128 columns is a 16-lane row of a wave and one of 32 four neighbouring lanes, whose
// maxima are DPP reductions without LDS.
#pragma once

#include "mm_front.h"

namespace mm {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two floats -> two BF16, round to nearest even, NaN kept.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 v = __builtin_convertvector((f32x2){lo, hi}, bf16x2);
  return __builtin_bit_cast(uint32_t, v);
}

// Largest of the bits of |v| over 4 neighbouring lanes / the 16 lanes of a row.  As unsigned
// integers magnitudes order as their values do, with infinity and NaN above every number.
__device__ __forceinline__ uint32_t max4(uint32_t m) {
  m = max(m, dpp<kXor1>(m));
  return max(m, dpp<kXor2>(m));
}
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  m = max4(m);
  m = max(m, dpp<kHalfMirror>(m));
  return max(m, dpp<kMirror>(m));
}

constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// Stores past the caches: rows that are written once, to places all over the memory or in larger amounts than the caches
// hold.
__device__ __forceinline__ void store16_nt(void* to, const uint4& v) {
  __builtin_nontemporal_store(v4i{(int)v.x, (int)v.y, (int)v.z, (int)v.w}, static_cast<v4i*>(to));
}

template <bool kF32>
__device__ __forceinline__ void store8(void* base, size_t elem, const float (&v)[8]) {
  if constexpr (kF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + elem) = pack_bf16x8(v);
  }
}

// The UE8M0 code of the smallest power of two >= r, for a finite r >= 0 in float64.
__device__ __forceinline__ uint32_t ue8m0_ceil64(double r) {
  const uint64_t u = __builtin_bit_cast(uint64_t, r);
  const int e = (int)(u >> 52) - 1023 + 127 + ((u & 0xFFFFFFFFFFFFFull) ? 1 : 0);
  return (uint32_t)min(max(e, 0), 254);
}

template <bool kF32>
__device__ __forceinline__ void store8_nt(void* base, size_t elem, const float (&v)[8]) {
  if constexpr (kF32) {
    float* p = static_cast<float*>(base) + elem;
    store16_nt(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
    store16_nt(p + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
  } else {
    store16_nt(static_cast<uint16_t*>(base) + elem, pack_bf16x8(v));
  }
}

// Eight values as loaded.
template <bool kF32>
struct Raw {
  uint4 v[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, size_t elem) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + elem * (kF32 ? 4 : 2));
    v[0] = p[0];
    if constexpr (kF32) v[1] = p[1];
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    if constexpr (kF32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(v[i].x);
        f[4 * i + 1] = __uint_as_float(v[i].y);
        f[4 * i + 2] = __uint_as_float(v[i].z);
        f[4 * i + 3] = __uint_as_float(v[i].w);
      }
    } else {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
};

}  // namespace mm
