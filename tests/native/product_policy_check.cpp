// The 8-bit product's choice of kernel and tile (csrc/mm_product_policy.h), compiled here by the host C++ compiler.  Built
// by tests/test_product_policy.py into a shared object and called through ctypes.
#include "mm_product_policy.h"

extern "C" {

int pp_variant(int64_t M, int64_t N, int64_t K, int64_t G) { return mm::product_variant(M, N, K, G); }
int pp_count() { return mm::kProductCount; }
int pp_n(int i) { return mm::kProductTiles[i].n; }
int pp_m(int i) { return mm::kProductTiles[i].m; }
int pp_most_blocks(int i) { return mm::kProductTiles[i].most_blocks; }
int64_t pp_workgroups(int i, int64_t M, int64_t N, int64_t G) { return mm::product_workgroups(mm::kProductTiles[i], M, N, G); }

}  // extern "C"
