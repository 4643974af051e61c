// The 8-bit product's search for a workgroup's tile (csrc/mm_product_policy.h), with the workgroup's threads one after the
// other, compiled by the host C++ compiler for tests/test_product_tiles.py.
#include "mm_product_policy.h"

extern "C" {

// How many threads find tile t, and what the last of them finds: its group, first row and rows.
int pt_find(const int32_t* offset, int G, int M, int m, int threads, int tiles, int t, int* out) {
  const int per = (G + threads - 1) / threads;
  uint32_t run = 0;
  int found = 0;
  for (int tid = 0; tid < threads; ++tid) {
    const int g0 = tid * per < G ? tid * per : G, g1 = g0 + per < G ? g0 + per : G;
    const uint32_t sum = mm::tiles_of(offset, g0, g1, M, m, tiles), before = run;
    run += sum;
    if ((uint32_t)t >= before && (uint32_t)t < run) {
      const mm::Tile r = mm::tile_among(offset, g0, g1, M, m, (uint32_t)t - before);
      out[0] = r.g, out[1] = r.m0, out[2] = r.rows;
      ++found;
    }
  }
  return found;
}

}  // extern "C"
