// The operators in front of the expert layer (residual RMS norm with 8-bit output, gate product,
// choice of experts): their arguments and host launchers, one translation unit each.
#pragma once

#include "mm_common.h"

namespace mm {

constexpr int kMaxGroups = 64;        // expert groups: one lane of a wave each
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

hipError_t launch_norm_quant(const NormArgs& a, hipStream_t s);
hipError_t launch_gate_logits(const GateArgs& a, hipStream_t s);
hipError_t launch_gate_topk(const TopkArgs& a, hipStream_t s);

}  // namespace mm
