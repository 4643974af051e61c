// Gate product: logits[t, e] = sum_h x[t, h] w[e, h] with BF16 MFMA, float32 sums.
//
// Weights are the MFMA's A operand (rows are experts) and tokens its B operand (columns), so a lane
// ends with four consecutive experts of one token and stores them as one float4.  Float32 weights
// are split into three BF16 terms of 8 significant bits each (w = hi + mid + lo exactly, by
// truncation) and multiplied by three MFMAs into the same sum.
#include "mm_front.h"

namespace mm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f mfma_bf16(const uint4& a, const uint4& b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The upper halves of two words: two BF16 by truncation.
__device__ __forceinline__ uint32_t upper_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ float truncated(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }

// Eight float32 values as three BF16 operands whose sum they are.
__device__ __forceinline__ void split3(const float (&v)[8], uint4 (&t)[3]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    t[p] = make_uint4(upper_halves(r[0], r[1]), upper_halves(r[2], r[3]), upper_halves(r[4], r[5]), upper_halves(r[6], r[7]));
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] -= truncated(r[i]);
  }
}

// One workgroup per tile of 16 experts x 16 tokens, four waves sharing K, joined through LDS.
template <bool kWF32>
__global__ __launch_bounds__(256) void k_gate(GateArgs a) {
  __shared__ v4f s_part[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, lg = lane >> 4;
  const int et = (a.E + 15) / 16;
  const long tiles = (long)et * ((a.T + 15) / 16);
  for (long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int e0 = (int)(tile % et) * 16, t0 = (int)(tile / et) * 16;
    const uint16_t* xr = a.x + (size_t)min(t0 + col, a.T - 1) * a.x_stride + 8 * lg;
    const size_t wr = (size_t)min(e0 + col, a.E - 1) * a.H + 8 * lg;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    for (int k = 32 * wave; k < a.H; k += 128) {
      const uint4 b = *reinterpret_cast<const uint4*>(xr + k);
      if constexpr (kWF32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.w) + wr + k);
        const float4 u = p[0], v = p[1];
        const float f[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        uint4 t[3];
        split3(f, t);
#pragma unroll
        for (int i = 0; i < 3; ++i) acc = mfma_bf16(t[i], b, acc);
      } else {
        acc = mfma_bf16(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.w) + wr + k), b, acc);
      }
    }
    s_part[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
      const v4f sum = (s_part[0][lane] + s_part[1][lane]) + (s_part[2][lane] + s_part[3][lane]);
      const int t = t0 + col, e = e0 + 4 * lg;
      if (t < a.T) {
        float* out = a.logits + (size_t)t * a.E + e;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < a.E) out[i] = sum[i];
      }
    }
    __syncthreads();                               // the parts are read before the next tile's are written
  }
}

}  // namespace

hipError_t launch_gate_logits(const GateArgs& a, hipStream_t s) {
  const long tiles = (long)((a.E + 15) / 16) * ((a.T + 15) / 16);
  const int grid = (int)(tiles < (1 << 20) ? tiles : (1 << 20));
  if (a.w_f32) hipLaunchKernelGGL((k_gate<true>), dim3(grid), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_gate<false>), dim3(grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace mm
