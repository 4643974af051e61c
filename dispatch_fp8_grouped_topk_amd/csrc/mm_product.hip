// 8-bit matrix product with a scale for each block of 128, by group of rows or dense:
//
//   y[m, n] = bf16( sum_b sx[m, b] sw[g, n / 128, b] sum_{k in b} x[m, k] w[g, n, k] )
//
// Weight rows are the MFMA's A operand and x's rows its B operand, so a lane ends with four consecutive columns of one
// row of y.  A 16x16x128 MFMA spans one block; its result is scaled and added to the float32 sums.
#include "mm_parts.h"
#include "mm_rows.h"

namespace mm {
namespace {

// The rows of group g, whatever the offsets hold.
__device__ __forceinline__ void group_rows(const ProductArgs& a, int g, int& lo, int& hi) {
  lo = 0;
  hi = a.M;
  if (a.offset) {
    lo = min(max(a.offset[g], 0), a.M);
    hi = min(max(a.offset[g + 1], lo), a.M);
  }
}

// Few rows a group: a workgroup takes 16 kRT weight rows of a group; its eight waves share K, wave w the blocks w, w + 8, ...
// straight from memory to registers, and their sums meet in LDS in a fixed order.
template <int kRT, int kCT>
__global__ __launch_bounds__(512) void k_product_small(ProductArgs a) {
  constexpr int kWaves = 8;
  __shared__ v4f sums[kWaves][kRT][kCT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lr = lane & 15, lg = lane >> 4;
  const int g = blockIdx.y, n0 = blockIdx.x * 16 * kRT, KB = a.K / 128;
  int lo, hi;
  group_rows(a, g, lo, hi);
  const uint8_t* w[kRT];
#pragma unroll
  for (int r = 0; r < kRT; ++r) w[r] = a.w + ((size_t)g * a.N + min(n0 + 16 * r + lr, a.N - 1)) * a.K;
  const float* sw = a.w_sf + ((size_t)g * ((a.N + 127) / 128) + n0 / 128) * KB;
  for (int64_t m0 = lo + (int64_t)blockIdx.z * 16 * kCT; m0 < hi; m0 += (int64_t)gridDim.z * 16 * kCT) {
    const uint8_t* x[kCT];
    const float* sx[kCT];
#pragma unroll
    for (int c = 0; c < kCT; ++c) {
      const int64_t row = min(m0 + 16 * c + lr, (int64_t)hi - 1);
      x[c] = a.x + row * a.x_stride;
      sx[c] = a.x_sf + row * KB;
    }
    v4f acc[kRT][kCT];
#pragma unroll
    for (int r = 0; r < kRT; ++r)
#pragma unroll
      for (int c = 0; c < kCT; ++c) acc[r][c] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int b = wave; b < KB; b += kWaves) {
      v8i A[kRT], B[kCT];
#pragma unroll
      for (int r = 0; r < kRT; ++r) A[r] = load_fp8_operand(w[r] + 128 * b, lg);
#pragma unroll
      for (int c = 0; c < kCT; ++c) B[c] = load_fp8_operand(x[c] + 128 * b, lg);
      const float s = sw[b];
#pragma unroll
      for (int c = 0; c < kCT; ++c) {
        const float sc = sx[c][b] * s;
#pragma unroll
        for (int r = 0; r < kRT; ++r) acc[r][c] += mfma_fp8(A[r], B[c]) * sc;
      }
    }
#pragma unroll
    for (int r = 0; r < kRT; ++r)
#pragma unroll
      for (int c = 0; c < kCT; ++c) sums[wave][r][c][lane] = acc[r][c];
    __syncthreads();
    for (int i = threadIdx.x; i < kRT * kCT * 64; i += 64 * kWaves) {
      const int l = i & 63, rc = i >> 6, r = rc / kCT, c = rc - r * kCT;
      v4f t = sums[0][r][c][l];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) t += sums[v][r][c][l];
      const int64_t row = m0 + 16 * c + (l & 15);
      const int n = n0 + 16 * r + 4 * (l >> 4);
      if (row < hi && n < a.N) {
        uint2 o;
        o.x = pack_bf16(t[0], t[1]);
        o.y = pack_bf16(t[2], t[3]);
        *reinterpret_cast<uint2*>(a.y + row * a.y_stride + n) = o;
      }
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_product(const ProductArgs& a, hipStream_t s) {
  const int per = (a.M + a.G - 1) / a.G;
  const int strips = a.offset ? std::min(64, (per + 63) / 64) : std::min(1024, (a.M + 63) / 64);
  hipLaunchKernelGGL((k_product_small<1, 4>), dim3((a.N + 15) / 16, a.G, strips), dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace mm
