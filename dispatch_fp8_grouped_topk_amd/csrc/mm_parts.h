// The layer in parts (tokens sorted by expert and back, the 8-bit product, the activation between two
// products): arguments and host launchers, one translation unit each for sorting, product and activation.
#pragma once

#include "mm_common.h"

namespace mm {

// ------------------------------------------------------------------------------------------ sort
// Batches of at most kSortSmallPairs pairs are sorted in one launch without workspace; larger ones in blocks of
// sort_block_pairs() pairs, at most kSortMaxBlocks of them.
constexpr int kSortSmallPairs = 4096, kSortChunk = 1024, kSortMaxBlocks = 1024;
constexpr int sort_block_pairs(int64_t P) {
  return (int)((P + (int64_t)kSortChunk * kSortMaxBlocks - 1) / ((int64_t)kSortChunk * kSortMaxBlocks)) * kSortChunk;
}
constexpr int sort_blocks(int64_t P) { return (int)((P + sort_block_pairs(P) - 1) / sort_block_pairs(P)); }

struct SortArgs {
  const void* x;             // [T, row_bytes], x_stride bytes apart, or NULL
  const uint32_t* x_sf;      // [T, sf_words] or NULL
  const int32_t* idx;        // [T, k]
  void* rows;                // [P, row_bytes]
  uint32_t* rows_sf;         // [P, sf_words]
  int32_t* src;              // [P]
  int32_t* pos;              // [T, k]
  int32_t* offset;           // [E + 1]
  int32_t* blk;              // workspace (large batches): [NB][E] pairs of each expert in each block, then those in
                             // earlier blocks
  int32_t* total;            // workspace: [E] pairs of each expert
  size_t x_stride;
  int T, k, E, P, NB, block_pairs;
  int row_bytes, sf_words;   // a row's 16-byte chunks times 16; its scales as 32-bit words
};

struct UnsortArgs {
  const void* rows;          // [R, H] bf16 | f32
  const int32_t* pos;        // [T, k]
  const float* w;            // [T, k] or NULL
  void* y;                   // [T, H], rows `stride` apart
  const void* dy;            // the gradient's: [T, H], rows `stride` apart
  void* d_rows;              // [R, H] or NULL
  float* d_w;                // [T, k] or NULL
  long stride;
  int T, H, k, R;
  int f32;
};

hipError_t launch_sort(const SortArgs& a, hipStream_t s);
hipError_t launch_unsort(const UnsortArgs& a, hipStream_t s);
hipError_t launch_unsort_backward(const UnsortArgs& a, hipStream_t s);

// --------------------------------------------------------------------------------------- product
constexpr int kMaxProductN = 1 << 20;
constexpr int64_t kMaxProductStride = 1 << 22;   // a tile's rows of x are addressed with 31-bit offsets

struct ProductArgs {
  const uint8_t* x;          // [M, K], rows x_stride apart
  const float* x_sf;         // [M, K/128]
  const uint8_t* w;          // [G, N, K]
  const float* w_sf;         // [G, ceil(N/128), K/128]
  const int32_t* offset;     // [G + 1] or NULL
  uint16_t* y;               // [M, N], rows y_stride apart
  long x_stride, y_stride;
  int M, N, K, G;
};

hipError_t launch_product(const ProductArgs& a, hipStream_t s);

// ------------------------------------------------------------------------------------ activation
struct ActArgs {
  const void* x;             // [M, I] | [M, 2I] bf16 | f32, rows x_stride apart
  const int32_t* num_valid;  // [1] or NULL
  uint8_t* q;                // [M, I] or NULL
  void* q_sf;                // [M, I/128] f32 | [M, I/32] UE8M0
  uint16_t* out;             // [M, I] bf16 or NULL
  const void* d_out;         // the gradient's: [M, I]
  void* d_x;                 // [M, 2I], rows x_stride apart
  long x_stride;
  int M, I;
  float clamp;               // <= 0: none
  int clamp_inputs;
  int swiglu, f32, per32;
  uint64_t by_row;           // factors that take the place of divisions (csrc/mm_act.hip sets them)
  uint32_t by_piece;
};

hipError_t launch_act_quant(const ActArgs& a, hipStream_t s);
hipError_t launch_act_backward(const ActArgs& a, hipStream_t s);

}  // namespace mm
