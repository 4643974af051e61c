// Which kernel and tile the gate product takes, by sizes and the weights' type.  No HIP headers: a plain C++ compiler
// can check it on the CPU.
#pragma once

#include <stdint.h>

namespace mm {

// Rows of a few tokens go to k_gate_rows as long as reading them again for each logit costs less than the
// tiles' K loop of fixed length.  Measured (us, rows with one token a workgroup, with two, tiles; H 7168, E 256):
// BF16 weights T 1 2.4, 2.7, 5.1; T 4 3.0, 3.0, 5.1; T 8 3.8, 3.7, 5.1; T 16 5.5, 4.9, 5.1; float32 T 1 2.5,
// 2.7, 6.9; T 4 3.4, 3.3, 7.0; T 8 4.6, 4.2, 6.9; T 16 7.5, 6.1, 6.9.  T 32, E 64, H 4096 3.5, 3.4, 4.4; with few
// experts the tiles win sooner: T 256, E 8, H 7168 6.3, 6.4, 5.0.
constexpr int64_t kRowsTokens = 64;
constexpr int64_t kRowsLogits = 2048;
constexpr int64_t kRowsSingle = 512;

// The tile sizes built (experts, tokens).  A workgroup fetches its rows of both operands once, at 40 to
// 50 bytes a clock and compute unit whatever the tile, so the time goes as the bytes of a tile's rows
// times the rounds its workgroups need on 256 compute units; the smallest product wins, of equal
// ones the smaller tile.  Measured (us, H 7168, E 256; the chosen tile, the next smaller, the next larger):
// BF16 weights T 1 (without k_gate_rows) 5.1, -, 5.7; T 128 7.4, 10.9, 8.3 (8 x 16); T 1024 13.6, 20.5, 17.8 (32 x 32); T 2048 18.4,
// 25.4, 23.2; T 4096 24.6, 34.9, 33.0; T 8192 49.6, 64.2, - (128 x 64); float32 weights T 1 6.7, -, 7.8;
// T 128 // 9.9, 15.3, 10.7 (8 x 16); T 1024 20.7, 27.8, 25.3; T 8192 86.9, 120.3, - (64 x 128).
struct GateTile {
  int e, t;
};
constexpr GateTile kGateTilesBf16[] = {{8, 8}, {8, 16}, {16, 16}, {16, 32}, {32, 32}, {64, 32}, {64, 64}, {128, 64}};
constexpr GateTile kGateTilesF32[] = {{8, 8}, {8, 16}, {16, 16}, {16, 32}, {32, 32}, {32, 64}, {64, 128}};

template <int kCount>
constexpr int gate_tile(const GateTile (&tiles)[kCount], int weight_bytes, int64_t T, int64_t E) {
  int best = 0;
  int64_t least = 0;
  for (int i = 0; i < kCount; ++i) {
    const GateTile t = tiles[i];
    const int64_t groups = ((E + t.e - 1) / t.e) * ((T + t.t - 1) / t.t);
    const int64_t cost = (groups + 255) / 256 * (t.e * weight_bytes + t.t * 2);
    if (i == 0 || cost < least) best = i, least = cost;
  }
  return best;
}

// Rows with one or two tokens a workgroup, or the tile's place in its list.
constexpr int kGateRowsSingle = -1, kGateRowsPair = -2;
constexpr int gate_variant(int64_t T, int64_t E, bool w_f32) {
  if (T <= kRowsTokens && T * E <= kRowsLogits) return T == 1 || T * E <= kRowsSingle ? kGateRowsSingle : kGateRowsPair;
  return w_f32 ? gate_tile(kGateTilesF32, 4, T, E) : gate_tile(kGateTilesBf16, 2, T, E);
}

}  // namespace mm
