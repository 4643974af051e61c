// Launch sizes of the 8-bit product (csrc/mm_product_policy.h), compiled by the host C++ compiler for
// tests/test_product_launches.py.
#include "mm_product_policy.h"

extern "C" {

int64_t pl_items(int i, int64_t M, int64_t N, int64_t G, int by_group) {
  return mm::product_items(mm::kProductTiles[i], M, N, G, by_group != 0);
}
int64_t pl_groups() { return mm::kProductGroups; }
int64_t pl_area() { return mm::kMaxProductArea; }

}  // extern "C"
