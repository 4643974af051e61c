// The gate product's choice of kernel and tile (csrc/mm_gate_policy.h), compiled here by the host C++ compiler.  Built
// by tests/test_gate_policy.py into a shared object and called through ctypes.
#include "mm_gate_policy.h"

extern "C" {

int gp_variant(int64_t T, int64_t E, int w_f32) { return mm::gate_variant(T, E, w_f32 != 0); }
int gp_tiles(int w_f32) {
  return w_f32 ? sizeof(mm::kGateTilesF32) / sizeof(mm::GateTile) : sizeof(mm::kGateTilesBf16) / sizeof(mm::GateTile);
}
int gp_tile_e(int w_f32, int i) { return w_f32 ? mm::kGateTilesF32[i].e : mm::kGateTilesBf16[i].e; }
int gp_tile_t(int w_f32, int i) { return w_f32 ? mm::kGateTilesF32[i].t : mm::kGateTilesBf16[i].t; }

}  // extern "C"
