// The activation between two products, with the 8-bit output that the next one takes, and its gradient.
//
//   s = 1 / (1 + exp(-g));  v = g s u, clamped;  per group of 128: sf = amax/448, q = E4M3(v / sf); per 32: the
//   UE8M0 code of the smallest power of two that holds amax/448
//   d_u = d g s,  d_g = d u s (1 + g (1 - s))
//
// One pass, eight columns a lane, nothing shared beyond 16 lanes, so the grid is flat over all pieces of all rows.  Bound by
// memory: 65536 x 2048 from BF16 with float scales (665 MB) takes 124 us, 5.3 TB/s; the gradient of 4093 x 1536 in float32
// (126 MB) 21.3 us, 5.9 TB/s, its stores past the caches (through them 25.3; the 8-bit rows, read next, gain nothing).
//
// Numerics: float32 throughout.  With e = exp(-|g|) in (0, 1] and r = 1 / (1 + e), s and 1 - s are r and e r or the other
// way round: neither overflows or cancels.  The hardware's exponential takes g log2(e), rounded: its relative error is
// at most 2^-17 (|g| 88; beyond, e is below float32's normal numbers) and 2^-21 for |g| up to 6.  Where that decides something that
// jumps, a UE8M0 code or whether a value lies inside the clamp, it is decided again in float64.
#include "mm_parts.h"
#include "mm_rows.h"

namespace mm {
namespace {

constexpr float kClose = 1.0f / 65536;           // twice the largest relative error of v

struct Sigmoid {
  float s, rest;                                 // s(g) and 1 - s(g)
};
__device__ __forceinline__ Sigmoid sigmoid(float g) {
  const float e = __expf(-fabsf(g)), r = __builtin_amdgcn_rcpf(1.0f + e);
  return g >= 0.f ? Sigmoid{r, e * r} : Sigmoid{e * r, r};
}

// v in [-c, c]; NaN stays NaN.
template <class T>
__device__ __forceinline__ T clamped(T v, T c) {
  return v > c ? c : v < -c ? -c : v;
}

__device__ __forceinline__ double swiglu64(float g, float u, float c, bool inputs) {
  const double gd = inputs ? clamped(g, c) : g, ud = inputs ? clamped(u, c) : u;
  const double v = gd / (1.0 + exp(-gd)) * ud;
  return c > 0.f && !inputs ? clamped(v, (double)c) : v;
}

// Rows that are looked at.
__device__ __forceinline__ int rows_used(const ActArgs& a) {
  return a.num_valid ? min(max(*a.num_valid, 0), a.M) : a.M;
}

template <bool kF32, bool kSwiglu, bool kPer32>
__global__ __launch_bounds__(256) void k_act_quant(ActArgs a) {
  const int cpt = a.I / 8;
  const int64_t total = (int64_t)rows_used(a) * cpt;
  const bool inputs = a.clamp > 0.f && a.clamp_inputs, output = a.clamp > 0.f && !a.clamp_inputs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / cpt;
    const int c = (int)(i - row * cpt);
    Raw<kF32> raw, raw_u;
    raw.load(a.x, (size_t)row * a.x_stride + 8 * c);
    if constexpr (kSwiglu) raw_u.load(a.x, (size_t)row * a.x_stride + a.I + 8 * c);
    float g[8], u[8], v[8];
    raw.values(g);
    if constexpr (kSwiglu) {
      raw_u.values(u);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        float gn = g[n], un = u[n];
        if (inputs) {
          gn = clamped(gn, a.clamp);
          un = clamped(un, a.clamp);
        }
        v[n] = gn * sigmoid(gn).s * un;
        if (output) v[n] = clamped(v[n], a.clamp);
      }
    } else {
#pragma unroll
      for (int n = 0; n < 8; ++n) v[n] = g[n];
    }
    const size_t at = (size_t)row * a.I + 8 * c;
    if (a.out) *reinterpret_cast<uint4*>(a.out + at) = pack_bf16x8(v);
    if (!a.q) continue;
    uint32_t m = 0;
#pragma unroll
    for (int n = 0; n < 8; ++n) m = max(m, mag(v[n]));
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
      if ((threadIdx.x & 15) == 0) static_cast<float*>(a.q_sf)[(size_t)row * (a.I / 128) + c / 16] = sf;
    } else {
      m = max4(m);
      const float r = __uint_as_float(m) * (1.0f / 448.0f);
      const uint32_t b = __float_as_uint(r), man = b & 0x7FFFFFu;
      uint32_t code = min((b >> 23) + 1, 254u);
      // kClose of the mantissa on either side of a power of two; the same in the four lanes of a group
      if (man <= 128 || man >= 0x7FFFFFu - 128 || b < 0x00800000u) {
        double d = 0.0;
#pragma unroll
        for (int n = 0; n < 8; ++n) d = fmax(d, fabs(kSwiglu ? swiglu64(g[n], u[n], a.clamp, inputs) : (double)g[n]));
        d = fmax(d, dpp<kXor1>(d));
        d = fmax(d, dpp<kXor2>(d));
        code = ue8m0_ceil64(d / 448.0);
      }
      if (m >= kInfBits) code = 255;
      const int up = 127 - (int)code;
#pragma unroll
      for (int n = 0; n < 8; ++n) v[n] = clamp448(__builtin_ldexpf(v[n], up));
      out.x = pack_fp8x4(v[0], v[1], v[2], v[3]);
      out.y = pack_fp8x4(v[4], v[5], v[6], v[7]);
      if (m >= kInfBits) out = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
      code |= dpp<kShl + 4>(code) << 8;            // lane 0 of the row: the row's four codes
      code |= dpp<kShl + 8>(code) << 16;
      if ((threadIdx.x & 15) == 0)
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.q_sf) + (size_t)row * (a.I / 32) + c / 4) = code;
    }
    *reinterpret_cast<uint2*>(a.q + at) = out;
  }
}

template <bool kF32>
__global__ __launch_bounds__(256) void k_act_backward(ActArgs a) {
  const int cpt = a.I / 8;
  const int64_t total = (int64_t)rows_used(a) * cpt;
  const bool inputs = a.clamp > 0.f && a.clamp_inputs, output = a.clamp > 0.f && !a.clamp_inputs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / cpt;
    const int c = (int)(i - row * cpt);
    const size_t at = (size_t)row * a.x_stride + 8 * c;
    Raw<kF32> rg, ru, rd;
    rg.load(a.x, at);
    ru.load(a.x, at + a.I);
    rd.load(a.d_out, (size_t)row * a.I + 8 * c);
    float g[8], u[8], d[8];
    rg.values(g);
    ru.values(u);
    rd.values(d);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      // what the clamp drops is selected, not multiplied by 0: the other factors may not be finite
      bool keep_g = !inputs || !(fabsf(g[n]) > a.clamp), keep_u = !inputs || !(fabsf(u[n]) > a.clamp);
      if (inputs) {
        g[n] = clamped(g[n], a.clamp);
        u[n] = clamped(u[n], a.clamp);
      }
      const Sigmoid s = sigmoid(g[n]);
      const float silu = g[n] * s.s;
      if (output) {
        const float v = fabsf(silu * u[n]);
        bool outside = v > a.clamp;
        if (fabsf(v - a.clamp) <= kClose * a.clamp) outside = fabs(swiglu64(g[n], u[n], 0.f, false)) > (double)a.clamp;
        if (outside) keep_g = keep_u = false;
      }
      const float du = d[n] * silu;
      g[n] = keep_g ? d[n] * u[n] * s.s * (1.0f + g[n] * s.rest) : 0.f;
      u[n] = keep_u ? du : 0.f;
    }
    store8_nt<kF32>(a.d_x, at, g);
    store8_nt<kF32>(a.d_x, at + a.I, u);
  }
}

unsigned pieces_grid(const ActArgs& a) {
  return (unsigned)std::min<int64_t>(((int64_t)a.M * (a.I / 8) + 255) / 256, 1 << 20);
}

template <bool kF32, bool kSwiglu>
void launch_quant(const ActArgs& a, hipStream_t s) {
  if (a.per32) hipLaunchKernelGGL((k_act_quant<kF32, kSwiglu, true>), dim3(pieces_grid(a)), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_act_quant<kF32, kSwiglu, false>), dim3(pieces_grid(a)), dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_act_quant(const ActArgs& a, hipStream_t s) {
  if (a.swiglu) a.f32 ? launch_quant<true, true>(a, s) : launch_quant<false, true>(a, s);
  else a.f32 ? launch_quant<true, false>(a, s) : launch_quant<false, false>(a, s);
  return hipGetLastError();
}

hipError_t launch_act_backward(const ActArgs& a, hipStream_t s) {
  if (a.f32) hipLaunchKernelGGL(k_act_backward<true>, dim3(pieces_grid(a)), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_act_backward<false>, dim3(pieces_grid(a)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace mm
