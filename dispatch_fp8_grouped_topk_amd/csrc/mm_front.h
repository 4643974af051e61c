// The operators in front of the expert layer (residual RMS norm with 8-bit output, gate product,
// choice of experts): their arguments and host launchers, one translation unit each.
#pragma once

#include "mm_common.h"

namespace mm {

constexpr int kMaxGroups = 64;        // expert groups: one lane of a wave each
constexpr int64_t kGateTokens = 1 << 23;   // tokens of one launch of the gate product
constexpr long kMaxGateStride = 1 << 22;  // the gate addresses a tile's rows of x with 31-bit offsets

struct NormArgs {
  const void* x;             // [T, H] bf16 | f32, rows x_stride apart
  const void* residual;      // [T, H] of x's type, rows residual_stride apart, or NULL
  const void* weight;        // [H] bf16 | f32
  void* residual_out;        // as residual, or NULL
  uint16_t* normed;          // [T, H] bf16, or NULL
  uint8_t* q;                // [T, H] E4M3, or NULL
  void* q_sf;                // [T, H/128] f32 | [T, H/32] UE8M0
  long x_stride, residual_stride;
  int T, H;
  float eps;
  int x_f32, w_f32;
  int per32;                 // 1: a UE8M0 scale per 32 columns; 0: a float scale per 128
};

struct GateArgs {
  const uint16_t* x;         // [T, H] bf16, rows x_stride apart
  const void* w;             // [E, H] bf16 | f32
  float* logits;             // [T, E]
  long x_stride;
  int T, H, E;
  int w_f32;
};

struct TopkArgs {
  const void* logits;        // [T, E] f32 | bf16, rows `stride` apart
  const float* bias;         // [E] or NULL
  const int32_t* num_valid;  // [1] or NULL
  int32_t* idx;              // [T, k + S]
  float* w;                  // [T, k + S]
  long stride;
  int T, E, k, S, G, KG;
  int group_top;
  int sigmoid, renorm, bf16;
  float scale, shared_weight;
};

// Lanes of a wave by DPP: v of the lane that kCtrl names (0 where there is none).
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
}
template <int kCtrl>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp<kCtrl>((uint32_t)u) | (uint64_t)dpp<kCtrl>((uint32_t)(u >> 32)) << 32);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;   // quad_perm, row_*mirror
constexpr int kBcast15 = 0x142, kBcast31 = 0x143, kShl = 0x100, kRor = 0x120;     // row_bcast, row_shl:n, row_ror:n

template <int kCtrl>
struct Ctrl {
  static constexpr int value = kCtrl;
};

// The sum / the largest over the 64 lanes, in lane 63.
__device__ __forceinline__ double wave_sum63(double v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  const double rows = dpp<kBcast15>(v);            // lane 15 -> row 1, lane 31 -> row 2, lane 47 -> row 3
  v += (threadIdx.x & 16) ? rows : 0.0;            // rows 1 and 3
  const double half = dpp<kBcast31>(v);            // lane 31 -> rows 2 and 3
  return v + ((threadIdx.x & 32) ? half : 0.0);
}
__device__ __forceinline__ float wave_sum63(float v) {
  const auto from = [](float u, auto ctrl) { return __uint_as_float(dpp<decltype(ctrl)::value>(__float_as_uint(u))); };
  v += from(v, Ctrl<kXor1>{});
  v += from(v, Ctrl<kXor2>{});
  v += from(v, Ctrl<kHalfMirror>{});
  v += from(v, Ctrl<kMirror>{});
  const float rows = from(v, Ctrl<kBcast15>{});
  v += (threadIdx.x & 16) ? rows : 0.f;
  const float half = from(v, Ctrl<kBcast31>{});
  return v + ((threadIdx.x & 32) ? half : 0.f);
}
__device__ __forceinline__ uint32_t wave_max63(uint32_t v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  v = max(v, dpp<kMirror>(v));
  v = max(v, dpp<kBcast15>(v));                    // lanes without a source read 0
  return max(v, dpp<kBcast31>(v));
}

hipError_t launch_norm_quant(const NormArgs& a, hipStream_t s);
hipError_t launch_gate_logits(const GateArgs& a, hipStream_t s);
hipError_t launch_gate_topk(const TopkArgs& a, hipStream_t s);

}  // namespace mm
