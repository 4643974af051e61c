// Residual addition, RMS norm and quantisation to the forward's 8-bit rows, one pass over each row:
// the row stays in registers between the sum of squares and the output.
//
//   h = x + residual;  r = 1 / sqrt(mean(h^2) + eps);  v = h r weight
//   per group of 128: sf = amax/448, q = E4M3(v / sf); per 32: the UE8M0 code of the smallest power
//   of two s with amax/s <= 448, q = E4M3(v / s)
//
// A workgroup takes a row; a thread holds chunks of 8 consecutive columns, chunk tid + i * blockDim.  A
// group of 128 columns is then one 16-lane row of a wave and a group of 32 four neighbouring lanes, so
// group maxima are DPP reductions without LDS.  H is a multiple of 128, so a 16-lane row is wholly in
// or out.
//
// Bound by memory: T 8192, H 7168 (BF16 rows and residual, all outputs, 530 MB) takes 100.8 us, 5.26 TB/s,
// against the 5.4 TB/s that a large copy reaches here.  A single row takes 3.4 us, of which an empty
// launch is 2.
//
// Numerics: sums of squares and r are float64 (no overflow for any float32 h, and the power-of-two
// scales below can be decided exactly); v is float32; each output is rounded once from it.  A UE8M0
// code jumps where amax/448 passes a power of two: where the float32 value lies within 16 units in
// the last place of one (its error is at most 5: one rounding each of |h w|, r and two products, up
// to two units each just above a power of two), the code is decided again in float64.
#include "mm_front.h"

namespace mm {
namespace {

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

// 1 / sqrt(m) for a positive float64: the hardware's estimate and two Newton steps.  A mean that is
// not finite gives NaN.
__device__ __forceinline__ double rsqrt64(double m) {
  double y = __builtin_amdgcn_rsq(m);
  y = y * (1.5 - 0.5 * m * y * y);
  y = y * (1.5 - 0.5 * m * y * y);
  return m < __builtin_inf() ? y : __builtin_nan("");
}

// The UE8M0 code of the smallest power of two >= r, for a finite r >= 0 in float64.
__device__ __forceinline__ uint32_t ue8m0_ceil64(double r) {
  const uint64_t u = __builtin_bit_cast(uint64_t, r);
  const int e = (int)(u >> 52) - 1023 + 127 + ((u & 0xFFFFFFFFFFFFFull) ? 1 : 0);
  return (uint32_t)min(max(e, 0), 254);
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

template <bool kXF32, bool kWF32, bool kPer32, int kNC>
__global__ __launch_bounds__(1024) void k_norm_quant(NormArgs a) {
  __shared__ double s_part[2][16];
  const int chunks = a.H / 8, tid = threadIdx.x, waves = blockDim.x / 64;
  const double inv_h = 1.0 / a.H;
  int parity = 0;
  for (int row = blockIdx.x; row < a.T; row += gridDim.x, parity ^= 1) {
    Raw<kXF32> x[kNC], r[kNC];
    Raw<kWF32> wt[kNC];
#pragma unroll
    for (int i = 0; i < kNC; ++i) {
      const int c = tid + i * blockDim.x;
      if (c >= chunks) continue;
      x[i].load(a.x, (size_t)row * a.x_stride + 8 * c);
      if (a.residual) r[i].load(a.residual, (size_t)row * a.residual_stride + 8 * c);
    }
#pragma unroll
    for (int i = 0; i < kNC; ++i) {                // asked for before the sum is known, used after it
      const int c = tid + i * blockDim.x;
      if (c < chunks) wt[i].load(a.weight, 8 * c);
    }
    float h[kNC][8];
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kNC; ++i) {
      const int c = tid + i * blockDim.x;
      if (c >= chunks) continue;
      x[i].values(h[i]);
      if (a.residual) {
        float f[8];
        r[i].values(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += f[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)h[i][j], (double)h[i][j], sum);
    }
    sum = wave_sum63(sum);
    if ((tid & 63) == 63) s_part[parity][tid >> 6] = sum;
    __syncthreads();                               // the other parity's slots may still be read
    sum = 0.0;
    for (int w = 0; w < waves; ++w) sum += s_part[parity][w];
    const double r64 = rsqrt64(sum * inv_h + (double)a.eps);
    const float r32 = (float)r64;
#pragma unroll
    for (int i = 0; i < kNC; ++i) {
      const int c = tid + i * blockDim.x;
      if (c >= chunks) continue;
      float w[8], v[8];
      wt[i].values(w);
      if (a.residual_out) store8<kXF32>(a.residual_out, (size_t)row * a.residual_stride + 8 * c, h[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = h[i][j] * r32 * w[j];
      const size_t at = (size_t)row * a.H + 8 * c;
      if (a.normed) *reinterpret_cast<uint4*>(a.normed + at) = pack_bf16x8(v);
      if (!a.q) continue;
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, mag(v[j]));
      uint2 out;
      if constexpr (!kPer32) {
        m = max16(m);
        const float amax = __uint_as_float(m);
        const float sf = m < kInfBits ? amax / 448.0f : __builtin_nanf("");
        const float inv = 448.0f / amax;
        out.x = e4m3_scaled4(v[0], v[1], v[2], v[3], inv, sf);
        out.y = e4m3_scaled4(v[4], v[5], v[6], v[7], inv, sf);
        if (sf == 0.f) out = make_uint2(0, 0);       // all zero, or below float32's range
        if (m >= kInfBits) out = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        if ((tid & 15) == 0) static_cast<float*>(a.q_sf)[(size_t)row * (a.H / 128) + c / 16] = sf;
      } else {
        m = max4(m);
        const float r = __uint_as_float(m) * (1.0f / 448.0f);
        const uint32_t u = __float_as_uint(r), man = u & 0x7FFFFFu;
        uint32_t code = min((u >> 23) + 1, 254u);
        if (man <= 16 || man >= 0x7FFFFFu - 16 || u < 0x00800000u) {      // uniform in the four lanes
          double d = 0.0;
#pragma unroll
          for (int j = 0; j < 8; ++j) d = fmax(d, fabs((double)h[i][j] * (double)w[j]));
          d = fmax(d, dpp<kXor1>(d));
          d = fmax(d, dpp<kXor2>(d));
          code = ue8m0_ceil64(d * r64 / 448.0);
        }
        if (m >= kInfBits) code = 255;
        const int up = 127 - (int)code;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = clamp448(__builtin_ldexpf(v[j], up));
        out.x = pack_fp8x4(v[0], v[1], v[2], v[3]);
        out.y = pack_fp8x4(v[4], v[5], v[6], v[7]);
        if (m >= kInfBits) out = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        code |= dpp<kShl + 4>(code) << 8;          // lane 0 of the row: the row's four codes
        code |= dpp<kShl + 8>(code) << 16;
        if ((tid & 15) == 0) *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.q_sf) + (size_t)row * (a.H / 32) + c / 4) = code;
      }
      *reinterpret_cast<uint2*>(a.q + at) = out;
    }
  }
}

// One chunk a thread as far as a workgroup's 1024 threads go, then two: fewer threads with four chunks each
// were slower at every size (us with 1, 2, 4 chunks, H 7168: T 1 3.4, 3.5, 4.5; T 128 4.3, 4.5, 5.5; T 8192
// 100.8, 105.2, 107.0), as more of a row's loads are under way and less follows the sum.
template <bool kXF32, bool kWF32, bool kPer32>
void launch(const NormArgs& a, hipStream_t s) {
  const int chunks = a.H / 8, grid = a.T < (1 << 20) ? a.T : (1 << 20);
  const int per = chunks <= 1024 ? 1 : 2, threads = ((chunks + per - 1) / per + 63) / 64 * 64;
  if (per == 1) hipLaunchKernelGGL((k_norm_quant<kXF32, kWF32, kPer32, 1>), dim3(grid), dim3(threads), 0, s, a);
  else hipLaunchKernelGGL((k_norm_quant<kXF32, kWF32, kPer32, 2>), dim3(grid), dim3(threads), 0, s, a);
}

}  // namespace

hipError_t launch_norm_quant(const NormArgs& a, hipStream_t s) {
  const int v = (a.x_f32 ? 4 : 0) | (a.w_f32 ? 2 : 0) | (a.per32 ? 1 : 0);
  switch (v) {
    case 0: launch<false, false, false>(a, s); break;
    case 1: launch<false, false, true>(a, s); break;
    case 2: launch<false, true, false>(a, s); break;
    case 3: launch<false, true, true>(a, s); break;
    case 4: launch<true, false, false>(a, s); break;
    case 5: launch<true, false, true>(a, s); break;
    case 6: launch<true, true, false>(a, s); break;
    default: launch<true, true, true>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace mm
