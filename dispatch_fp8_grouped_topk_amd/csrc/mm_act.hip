// The activation between two products, with the 8-bit output that the next one takes, and its gradient.
//
//   s = 1 / (1 + exp(-g));  v = g s u, clamped;  per group of 128: sf = amax/448, q = E4M3(v / sf); per 32: the
//   UE8M0 code of the smallest power of two that holds amax/448
//   d_u = d g s,  d_g = d u s (1 + g (1 - s))
//
// One pass, eight columns a lane, nothing shared beyond 16 lanes, so the grid is flat over all pieces of all rows.  Bound by
// memory: 65536 x 2048 from BF16 with float scales (665 MB) takes 123 us, 5.4 TB/s; the gradient of 4093 x 1536 in float32
// (126 MB) 21.1 us, 6.0 TB/s, its stores past the caches (through them 25.3; the 8-bit rows, read next, gain nothing).
//
// Numerics: float32 throughout.  With e = exp(-|g|) in (0, 1] and r = 1 / (1 + e), s and 1 - s are r and e r or the other
// way round: neither overflows or cancels.  |g| log2(e) is taken in two parts, the product and what its rounding left: in one
// part it would cost |g| half steps of e.  v is within 9 half steps of float32 then (2^-24 of the value each).  Beyond
// |g| 86, where e may be no normal number, it is kept as f 2^n and the power applied to the other factor.  Where an error
// decides something that jumps, a UE8M0 code or whether a value lies inside the clamp, it is decided again in float64.
#include <type_traits>

#include "mm_parts.h"
#include "mm_rows.h"

namespace mm {
namespace {

// Float64 decides within kClose of a border, thirty times v's error, and kSmall, twice what v may be off by where float32 has
// few bits left.
constexpr float kClose = 1.0f / 65536, kSmall = 0x1p-140f;
constexpr float kFarGate = 86.f;                 // exp(-86) is still a normal number

// e = exp(-|g|) = f 2^n (n 0 unless kFar) and r = 1 / (1 + e).  A NaN stays one in what g is multiplied with.
struct Sigmoid {
  float r, e, f;
  int n;
};
template <bool kFar>
__device__ __forceinline__ Sigmoid sigmoid(float g) {
  constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;      // log2(e)
  const float a = kFar ? fminf(fabsf(g), 400.f) : fabsf(g);     // 2^-577 is 0 times any float
  const float t = a * kHi;
  Sigmoid s;
  if constexpr (kFar) {
    const float whole = __builtin_rintf(t);
    s.f = __builtin_amdgcn_exp2f(__builtin_fmaf(-a, kLo, __builtin_fmaf(-a, kHi, whole)));
    s.n = -(int)whole;
    s.e = __builtin_ldexpf(s.f, s.n);
  } else {
    const float p = __builtin_amdgcn_exp2f(-t), rest = __builtin_fmaf(a, kLo, __builtin_fmaf(a, kHi, -t));
    s.e = s.f = __builtin_fmaf(p, rest * -0.693147181f, p);      // 2^-rest to first order: rest is below 2^-17
    s.n = 0;
  }
  const float d = 1.0f + s.e, r = __builtin_amdgcn_rcpf(d);
  s.r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
  return s;
}

// x s(g)
template <bool kFar>
__device__ __forceinline__ float times_sigmoid(float x, float g, const Sigmoid& s) {
  if constexpr (kFar) return (g < 0.f ? __builtin_ldexpf(x, s.n) * s.f : x) * s.r;
  return x * (g < 0.f ? s.e * s.r : s.r);
}
// x silu(g)
template <bool kFar>
__device__ __forceinline__ float times_silu(float x, float g, const Sigmoid& s) {
  if constexpr (kFar) return (g < 0.f ? __builtin_ldexpf(x, s.n) * s.f : x) * (g * s.r);
  return g * (g < 0.f ? s.e * s.r : s.r) * x;
}

// Gates far out are taken again by themselves, so that a value depends on its own inputs alone.
__device__ __forceinline__ bool far_out(float g) { return fabsf(g) > kFarGate; }
__device__ __forceinline__ bool any_far(const float (&g)[8]) {
  float m = 0.f;
#pragma unroll
  for (int n = 0; n < 8; ++n) m = fmaxf(m, fabsf(g[n]));
  return far_out(m);
}

// v in [-c, c]; NaN stays NaN.
template <class T>
__device__ __forceinline__ T clamped(T v, T c) {
  return v > c ? c : v < -c ? -c : v;
}

__device__ __forceinline__ void clamp_all(float (&v)[8], float c) {
#pragma unroll
  for (int n = 0; n < 8; ++n) v[n] = clamped(v[n], c);
}

__device__ __forceinline__ double swiglu64(float g, float u, float c, bool inputs) {
  const double gd = inputs ? clamped(g, c) : g, ud = inputs ? clamped(u, c) : u;
  const double v = gd / (1.0 + exp(-gd)) * ud;
  return c > 0.f && !inputs ? clamped(v, (double)c) : v;
}

// Piece 256 b + threadIdx.x of eight columns among those of all rows: its row and its place there, without a division in
// 64 bits (about a hundred instructions a thread: 65536 x 2048 150 -> 145 us where arithmetic was the bound).  A row has 16 j pieces, so b starts in row 16 b / j: the high half of
// 16 b ceil(2^64 / j), exact as 16 b j < 2^64; from there less than 2304 pieces are counted, the high part of a product with
// ceil(2^24 / 16 j), exact as 2304 * 2048 < 2^24.
struct Piece {
  int64_t row;
  int c;
};
__device__ __forceinline__ Piece piece(const ActArgs& a, uint64_t b, int cpt) {
  const uint64_t row = a.by_row ? __umul64hi(16 * b, a.by_row) : 16 * b;
  const uint32_t c = (uint32_t)(256 * b - row * (uint32_t)cpt) + threadIdx.x, more = c * a.by_piece >> 24;
  return {(int64_t)(row + more), (int)(c - more * (uint32_t)cpt)};
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
  for (uint64_t b = blockIdx.x; (int64_t)(256 * b + threadIdx.x) < total; b += gridDim.x) {
    const auto [row, c] = piece(a, b, cpt);
    Raw<kF32> raw, raw_u;
    raw.load(a.x, (size_t)row * a.x_stride + 8 * c);
    if constexpr (kSwiglu) raw_u.load(a.x, (size_t)row * a.x_stride + a.I + 8 * c);
    float g[8], u[8], v[8];
    raw.values(g);
    if constexpr (kSwiglu) {
      raw_u.values(u);
      if (inputs) clamp_all(g, a.clamp), clamp_all(u, a.clamp);
#pragma unroll
      for (int n = 0; n < 8; ++n) v[n] = times_silu<false>(u[n], g[n], sigmoid<false>(g[n]));
      if (any_far(g)) {
#pragma unroll
        for (int n = 0; n < 8; ++n)
          if (far_out(g[n])) v[n] = times_silu<true>(u[n], g[n], sigmoid<true>(g[n]));
      }
      if (output) clamp_all(v, a.clamp);
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
      // kClose on either side of a power of two: 128 steps above it, 256 of half the size below; below float32's normal numbers
      // always.  The same in the four lanes of a group.
      if (man <= 128 || man >= 0x800000u - 256 || b < 0x00800000u) {
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

// kClamp: none, of the inputs, of the output; an instance of its own keeps the float64 decision's registers out of the others.
enum Clamp { kClampNone, kClampInputs, kClampOutput };
template <bool kF32, Clamp kClamp>
__global__ __launch_bounds__(256) void k_act_backward(ActArgs a) {
  const int cpt = a.I / 8;
  const int64_t total = (int64_t)rows_used(a) * cpt;
  for (uint64_t b = blockIdx.x; (int64_t)(256 * b + threadIdx.x) < total; b += gridDim.x) {
    const auto [row, c] = piece(a, b, cpt);
    const size_t at = (size_t)row * a.x_stride + 8 * c;
    Raw<kF32> rg, ru, rd;
    rg.load(a.x, at);
    ru.load(a.x, at + a.I);
    rd.load(a.d_out, (size_t)row * a.I + 8 * c);
    float g[8], u[8], d[8];
    rg.values(g);
    ru.values(u);
    rd.values(d);
    // what the clamp drops is selected, not multiplied by 0: the other factors may not be finite
    uint32_t drop_g = 0, drop_u = 0;
    if constexpr (kClamp == kClampInputs) {
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        drop_g |= (uint32_t)(fabsf(g[n]) > a.clamp) << n;
        drop_u |= (uint32_t)(fabsf(u[n]) > a.clamp) << n;
      }
      clamp_all(g, a.clamp), clamp_all(u, a.clamp);
    }
    float d_g[8], d_u[8], v[8];
    const auto gradient = [&](int n, auto far) {
      constexpr bool kFar = decltype(far)::value;
      const Sigmoid s = sigmoid<kFar>(g[n]);
      const float rest = g[n] < 0.f ? s.r : s.e * s.r;
      d_g[n] = times_sigmoid<kFar>(d[n] * u[n], g[n], s) * __builtin_fmaf(g[n], rest, 1.0f);
      d_u[n] = times_silu<kFar>(d[n], g[n], s);
      if constexpr (kClamp == kClampOutput) v[n] = fabsf(times_silu<kFar>(u[n], g[n], s));
    };
#pragma unroll
    for (int n = 0; n < 8; ++n) gradient(n, std::false_type{});
    if (any_far(g)) {
#pragma unroll
      for (int n = 0; n < 8; ++n)
        if (far_out(g[n])) gradient(n, std::true_type{});
    }
    if constexpr (kClamp == kClampOutput) {
      // near the largest numbers near_hi is infinite, and so may v be
      const float near_lo = __builtin_fmaf(a.clamp, -kClose, a.clamp) - kSmall;
      const float near_hi = __builtin_fmaf(a.clamp, kClose, a.clamp) + kSmall;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        bool outside = v[n] > a.clamp;
        if (v[n] >= near_lo && !(v[n] > near_hi)) outside = fabs(swiglu64(g[n], u[n], 0.f, false)) > (double)a.clamp;
        drop_g |= (uint32_t)outside << n;
      }
      drop_u = drop_g;
    }
    if constexpr (kClamp != kClampNone) {
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        d_g[n] = drop_g >> n & 1 ? 0.f : d_g[n];
        d_u[n] = drop_u >> n & 1 ? 0.f : d_u[n];
      }
    }
    store8_nt<kF32>(a.d_x, at, d_g);
    store8_nt<kF32>(a.d_x, at + a.I, d_u);
  }
}

ActArgs with_pieces(ActArgs a) {
  a.by_row = a.I == 128 ? 0 : ~0ull / (unsigned)(a.I / 128) + 1;       // 2^64 itself does not fit
  a.by_piece = ((1u << 24) + a.I / 8 - 1) / (a.I / 8);
  return a;
}

unsigned pieces_grid(const ActArgs& a) {
  return (unsigned)std::min<int64_t>(((int64_t)a.M * (a.I / 8) + 255) / 256, 1 << 20);
}

template <bool kF32, bool kSwiglu>
void launch_quant(const ActArgs& a, hipStream_t s) {
  if (a.per32) hipLaunchKernelGGL((k_act_quant<kF32, kSwiglu, true>), dim3(pieces_grid(a)), dim3(256), 0, s, with_pieces(a));
  else hipLaunchKernelGGL((k_act_quant<kF32, kSwiglu, false>), dim3(pieces_grid(a)), dim3(256), 0, s, with_pieces(a));
}

template <bool kF32>
void launch_backward(const ActArgs& a, hipStream_t s) {
  const dim3 grid(pieces_grid(a)), threads(256);
  if (!(a.clamp > 0.f)) hipLaunchKernelGGL((k_act_backward<kF32, kClampNone>), grid, threads, 0, s, with_pieces(a));
  else if (a.clamp_inputs) hipLaunchKernelGGL((k_act_backward<kF32, kClampInputs>), grid, threads, 0, s, with_pieces(a));
  else hipLaunchKernelGGL((k_act_backward<kF32, kClampOutput>), grid, threads, 0, s, with_pieces(a));
}

}  // namespace

hipError_t launch_act_quant(const ActArgs& a, hipStream_t s) {
  if (a.swiglu) a.f32 ? launch_quant<true, true>(a, s) : launch_quant<false, true>(a, s);
  else a.f32 ? launch_quant<true, false>(a, s) : launch_quant<false, false>(a, s);
  return hipGetLastError();
}

hipError_t launch_act_backward(const ActArgs& a, hipStream_t s) {
  a.f32 ? launch_backward<true>(a, s) : launch_backward<false>(a, s);
  return hipGetLastError();
}

}  // namespace mm
