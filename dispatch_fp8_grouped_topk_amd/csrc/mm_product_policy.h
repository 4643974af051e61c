// Which kernel and tile the 8-bit product takes, by sizes.  No HIP headers: a plain C++ compiler can check it on the CPU.
#pragma once

#include <stdint.h>

namespace mm {

// The instances built: a workgroup's weight rows and rows of x, and what its time goes by, fitted (us) to the times of
// every instance at 72 dense sizes (M 1 to 8192; N, K of 512 x 512, 512 x 7168, 2048 x 2048, 4096 x 7168, 7168 x 2048,
// 8192 x 512) to within 7 to 16% in the mean: per round of 256 workgroups a fixed part and one for each of the K/128 blocks.
// The first kProductSplit share K among a workgroup's waves (k_product_split, block time of all its waves together), the
// others share the tile (k_product_large; of {128, 64} the second shares K as well).  The smallest sum wins; over those sizes and 30 more by 4 to 256 groups the
// choice takes 2.7% longer than the best instance in the mean.  Both sides of some borders (us, K 7168, N 4096):
// M 16 {16, 16} 7.7, {32, 32} 8.5; M 128 {64, 32} 12.5, {64, 64} 17.4; M 256 {64, 64} 18.2, {128, 64} 24.9; M 512 {128, 64}
// 25.0, {64, 64} 34.4; M 1024 {128, 128} 39.4, {128, 64} 52.3; M 2048 {256, 128} 60.4, {256, 256} 85.4; M 4096 {256, 256} 103,
// {256, 128} 118.
struct ProductTile {
  int n, m;
  float fixed, block;        // us a round, us a round and block
  int most_blocks;           // of K that its LDS holds the scales of
};
constexpr ProductTile kProductTiles[] = {
    {16, 16, 1.9f, .049f, 128}, {16, 32, 1.75f, .073f, 128}, {32, 32, 1.8f, .101f, 128}, {64, 32, 2.3f, .133f, 128},
    {64, 64, 3.0f, .203f, 112}, {128, 64, 1.75f, .387f, 128}, {128, 64, 2.4f, .37f, 128}, {128, 128, 2.5f, .498f, 128},
    {256, 64, 2.5f, .518f, 128}, {256, 128, 3.3f, .724f, 128}, {256, 256, 3.9f, 1.27f, 128}};
constexpr int kProductCount = sizeof(kProductTiles) / sizeof(kProductTiles[0]), kProductSplit = 5;

// Most workgroups of a launch, whose threads are counted in 32 bits (512 each).  More are launched in parts; only the largest
// tile can need that (4096 rows by 1024 groups of 2^20 x 128 weights), the others are passed over then.
constexpr int64_t kProductGroups = 1 << 22;

// Least num_rows * n that is refused: below it a launch's items (product_items) fit 31 bits.
constexpr int64_t kMaxProductArea = (int64_t)1 << 45;

constexpr int64_t up_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Items of a launch, a workgroup each: every slab of weight rows and every tile that the groups may be cut into, with rows or
// without.
constexpr int64_t product_tiles(const ProductTile& t, int64_t M, int64_t G, bool by_group) {
  const int64_t whole = up_div(M, t.m);
  return !by_group ? whole : M < whole + G ? M : whole + G;
}
constexpr int64_t product_items(const ProductTile& t, int64_t M, int64_t N, int64_t G, bool by_group) {
  return up_div(N, t.n) * product_tiles(t, M, G, by_group);
}

// The rows of group g among M, whatever the offsets hold (NULL: all of them).
struct GroupRows {
  int lo, hi;
};
constexpr GroupRows group_rows(const int32_t* offset, int g, int M) {
  if (!offset) return GroupRows{0, M};
  const int from = offset[g] < 0 ? 0 : offset[g], lo = from < M ? from : M;
  const int to = offset[g + 1] < lo ? lo : offset[g + 1];
  return GroupRows{lo, to < M ? to : M};
}
// The tiles of m rows of groups [g0, g1), `tiles` at most: a launch has no more, and groups whose offsets ascend have no
// more.  Where they descend the true number may pass 32 bits; 512 times this one does not, so each tile has one finder.
constexpr uint32_t tiles_of(const int32_t* offset, int g0, int g1, int M, int m, int tiles) {
  uint32_t sum = 0;
  for (int g = g0; g < g1; ++g) {
    const GroupRows r = group_rows(offset, g, M);
    sum += (uint32_t)(r.hi - r.lo + m - 1) / (uint32_t)m;
  }
  return sum < (uint32_t)tiles ? sum : (uint32_t)tiles;
}
// The group and rows of the k-th of those tiles.
struct Tile {
  int g, m0, rows;
};
constexpr Tile tile_among(const int32_t* offset, int g0, int g1, int M, int m, uint32_t k) {
  for (int g = g0; g < g1; ++g) {
    const GroupRows r = group_rows(offset, g, M);
    const uint32_t n = (uint32_t)(r.hi - r.lo + m - 1) / (uint32_t)m;
    if (k < n) {
      const int m0 = r.lo + (int)k * m;
      return Tile{g, m0, r.hi - m0 < m ? r.hi - m0 : m};
    }
    k -= n;
  }
  return Tile{0, 0, 0};
}

// Workgroups that have rows: the rows of G groups are not known here and taken as uneven, each group's last tile as
// about half full.
constexpr int64_t product_workgroups(const ProductTile& t, int64_t M, int64_t N, int64_t G) {
  const int64_t active = G < M ? G : M;
  const int64_t tiles = G == 1 ? up_div(M, t.m) : active + up_div(M * M, (M + active * t.m) * t.m);
  return up_div(N, t.n) * tiles;
}

constexpr int product_variant(int64_t M, int64_t N, int64_t K, int64_t G) {
  int best = kProductCount - 1;
  float least = 0.f;
  for (int i = 0; i < kProductCount; ++i) {
    const ProductTile& t = kProductTiles[i];
    const int64_t w = product_workgroups(t, M, N, G), most = up_div(N, t.n) * (up_div(M, t.m) + G);
    if (K / 128 > t.most_blocks || (i + 1 < kProductCount && most > kProductGroups)) continue;
    const float cost = (float)up_div(w, 256) * (t.fixed + (float)(K / 128) * t.block);
    if (least == 0.f || cost < least) best = i, least = cost;
  }
  return best;
}

}  // namespace mm
