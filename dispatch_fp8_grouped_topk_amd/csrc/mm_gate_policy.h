// Which kernel and tile the gate product takes, by sizes and the weights' type.  No HIP headers: a plain C++ compiler
// can check it on the CPU.
#pragma once

#include <stdint.h>

namespace mm {

// Rows of a few tokens go to k_gate_rows as long as reading them again for each logit costs less than the
// tiles' K loop of fixed length.  Measured (us, rows with one token a workgroup, with two, tiles; H 7168, E 256):
// BF16 weights T 1 2.3, 2.5, 5.0; T 4 2.9, 2.9, 5.0; T 8 3.7, 3.5, 5.0; T 16 5.7, 4.9, 5.0; float32 T 1 2.3,
// 2.5, 6.8; T 4 3.2, 3.1, 6.9; T 8 4.5, 4.0, 6.8; T 16 7.3, 5.8, 6.9.  At T 8 the same holds for H 1024 (BF16 3.1, 3.0,
// 3.5; float32 3.0, 2.9, 3.8), H 4096 (3.3, 3.1, 4.2; 3.4, 3.2, 5.3) and H 16384 (6.2, 5.4, 7.1; 9.9, 7.9, 11.8), so the
// rule does not ask for H.  T 32, E 64, H 4096 3.2, 3.1, 4.2; with few experts the tiles win sooner: T 256, E 8,
// H 7168 6.1, 6.3, 5.0.
constexpr int64_t kRowsTokens = 64;
constexpr int64_t kRowsLogits = 2048;
constexpr int64_t kRowsSingle = 512;

// The tile sizes built (experts, tokens).  A workgroup fetches its rows of both operands once, at 40 to
// 50 bytes a clock and compute unit whatever the tile, so the time goes as the bytes of a tile's rows
// times the rounds its workgroups need on 256 compute units; the smallest product wins, of equal
// ones the smaller tile.  Measured (us, H 7168, E 256; the chosen tile, the next smaller, the next larger):
// BF16 weights T 128 7.2, 10.4, 8.0 (8 x 16); T 1024 13.3, 20.2, 17.5 (32 x 32); T 2048 18.0, 25.0, 23.0 (64 x 32);
// T 4096 24.0, 34.3, 32.4 (64 x 64); T 8192 47.9, 64.0, - (128 x 64); float32 weights T 128 9.0, 14.8, 10.3 (8 x 16);
// T 1024 19.8, 27.2, 24.5 (32 x 32); T 8192 82.9, 119, - (64 x 128).
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
