// C ABI of libmegamoe: argument validation, workspace carving and the launch sequence.
// No allocation, no synchronisation: every kernel is enqueued on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include "mega_moe.h"
#include "mm_common.h"
#include "mm_front.h"
#include "mm_parts.h"
#include "mm_product_policy.h"

#define MM_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

struct Layout {
  size_t hdr, count, offset, blk, blk_inv, pair_pos, pool_src, w_pool, tiles_s, tiles_l, x_sf_pool,
      inter_q, inter_sf, slot, tile_done, total;
  int P, NB, max_tiles_s, max_tiles_l;
};

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

int check_problem(const mega_moe_problem* p) {
  if (!p) return MEGA_MOE_ERR_NULL_POINTER;
  if (p->num_tokens < 0) return MEGA_MOE_ERR_INVALID_ARG;
  if (p->hidden <= 0 || p->hidden % 128 || p->hidden > 16384) return MEGA_MOE_ERR_INVALID_ARG;
  if (p->intermediate <= 0 || p->intermediate % 128 || p->intermediate > 16384) return MEGA_MOE_ERR_INVALID_ARG;
  if (p->num_experts < 1 || p->num_experts > mm::kMaxExperts) return MEGA_MOE_ERR_INVALID_ARG;
  if (p->topk < 1 || p->topk > mm::kMaxTopk) return MEGA_MOE_ERR_INVALID_ARG;
  if (p->recipe != MEGA_MOE_RECIPE_FP8_B128 && p->recipe != MEGA_MOE_RECIPE_MXFP4W_B32 &&
      p->recipe != MEGA_MOE_RECIPE_MXFP8_B32)
    return MEGA_MOE_ERR_INVALID_ARG;
  if (std::isnan(p->swiglu_clamp) || p->swiglu_clamp < 0.f) return MEGA_MOE_ERR_INVALID_ARG;
  if (p->flags & ~(MEGA_MOE_FLAG_TILE_MASK | MEGA_MOE_FLAG_CLAMP_INPUTS | MEGA_MOE_FLAG_PRECISE_SILU |
                   MEGA_MOE_FLAG_WEIGHT_SF_KMAJOR | MEGA_MOE_FLAG_INTER_SF64 | MEGA_MOE_FLAG_FUSED |
                   MEGA_MOE_FLAG_WEIGHT_E2M1_PAIRED))
    return MEGA_MOE_ERR_INVALID_ARG;
  // the row-pair weight layout exists for the E2M1 weights only
  if ((p->flags & MEGA_MOE_FLAG_WEIGHT_E2M1_PAIRED) && p->recipe != MEGA_MOE_RECIPE_MXFP4W_B32)
    return MEGA_MOE_ERR_INVALID_ARG;
  // the fused forward runs the large-M GEMMs only
  if ((p->flags & MEGA_MOE_FLAG_FUSED) && (p->flags & MEGA_MOE_FLAG_TILE_MASK) == MEGA_MOE_FLAG_TILE_SMALL)
    return MEGA_MOE_ERR_INVALID_ARG;
  // per-64 float intermediate scales exist for the float-scale recipe only
  if ((p->flags & MEGA_MOE_FLAG_INTER_SF64) && p->recipe != MEGA_MOE_RECIPE_FP8_B128)
    return MEGA_MOE_ERR_INVALID_ARG;
  // the K-major weight-scale layout exists for the per-32 (UE8M0) recipes only
  if ((p->flags & MEGA_MOE_FLAG_WEIGHT_SF_KMAJOR) && p->recipe == MEGA_MOE_RECIPE_FP8_B128)
    return MEGA_MOE_ERR_INVALID_ARG;
  if ((p->flags & MEGA_MOE_FLAG_TILE_MASK) == MEGA_MOE_FLAG_TILE_MASK) return MEGA_MOE_ERR_INVALID_ARG;
  if (p->num_tokens * (int64_t)p->topk > (int64_t)(INT_MAX / 2)) return MEGA_MOE_ERR_INVALID_ARG;
  return MEGA_MOE_OK;
}

Layout make_layout(const mega_moe_problem* p) {
  Layout L{};
  const size_t T = (size_t)p->num_tokens, H = p->hidden, I = p->intermediate, E = p->num_experts;
  const size_t P = T * (size_t)p->topk;
  L.P = (int)P;
  L.NB = (int)((P + mm::kRouteBlock - 1) / mm::kRouteBlock);
  const size_t ts = P ? std::min(P, (P + mm::kSmallRows - 1) / mm::kSmallRows + E) : 0;
  const size_t tl = P ? std::min(P, (P + mm::kLargeRows - 1) / mm::kLargeRows + E) : 0;
  L.max_tiles_s = (int)ts;
  L.max_tiles_l = (int)tl;
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t r = o; o = align256(o + bytes); return r; };
  L.hdr = take(mm::kHdrWords * 4);
  L.count = take(E * 4);
  L.offset = take((E + 1) * 4);
  L.blk = take((size_t)L.NB * E * 4);
  L.blk_inv = take((size_t)L.NB * 4);
  L.pair_pos = take(P * 4);
  L.pool_src = take(P * 4);
  L.w_pool = take(P * 4);
  L.tiles_s = take(ts * 8);
  L.tiles_l = take(tl * 8);
  L.x_sf_pool = take(P * (H / 128) * 4);
  L.inter_q = take(P * I);
  const size_t inter_groups = (p->flags & MEGA_MOE_FLAG_INTER_SF64) ? I / 64 : I / 128;
  L.inter_sf = take(p->recipe == MEGA_MOE_RECIPE_FP8_B128 ? P * inter_groups * 4 : P * (I / 32));
  L.slot = take(P * H * 2);
  L.tile_done = take((tl + 1) * 4);
  L.total = o;
  return L;
}

// Per-device "is gfx950" cache: 0 unknown, 1 yes, 2 no.
std::atomic<int> g_arch_ok[64];

int check_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return MEGA_MOE_ERR_HIP;
  if (dev < 0 || dev >= 64) return MEGA_MOE_ERR_UNSUPPORTED_DEVICE;
  int st = g_arch_ok[dev].load(std::memory_order_relaxed);
  if (st == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MEGA_MOE_ERR_HIP;
    st = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_arch_ok[dev].store(st, std::memory_order_relaxed);
  }
  return st == 1 ? MEGA_MOE_OK : MEGA_MOE_ERR_UNSUPPORTED_DEVICE;
}

// Per-device compute-unit count (0 = not yet queried).
std::atomic<int> g_num_cus[64];

int device_cus() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
  int n = g_num_cus[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
    g_num_cus[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

inline bool misaligned(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) != 0; }

}  // namespace

MM_EXPORT int mega_moe_abi_version(void) { return MEGA_MOE_ABI_VERSION; }

MM_EXPORT const char* mega_moe_strerror(int status) {
  switch (status) {
    case MEGA_MOE_OK: return "ok";
    case MEGA_MOE_ERR_INVALID_ARG: return "invalid argument (a problem field is out of range)";
    case MEGA_MOE_ERR_NULL_POINTER: return "a required pointer is NULL";
    case MEGA_MOE_ERR_MISALIGNED: return "a pointer is not 16-byte aligned";
    case MEGA_MOE_ERR_WORKSPACE_TOO_SMALL: return "workspace smaller than mega_moe_workspace_size()";
    case MEGA_MOE_ERR_UNSUPPORTED_DEVICE: return "the current device is not gfx950 (MI355X)";
    case MEGA_MOE_ERR_HIP: return "a HIP runtime call or kernel launch failed";
    case MEGA_MOE_ERR_SCRATCH_TOO_SMALL:
      return "the problem needs more workspace than the static scratch of mega_moe_forward_noalloc (32 MiB)";
    default: return "unknown status";
  }
}

MM_EXPORT int mega_moe_workspace_size(const mega_moe_problem* p, size_t* bytes_out) {
  const int st = check_problem(p);
  if (st) return st;
  if (!bytes_out) return MEGA_MOE_ERR_NULL_POINTER;
  *bytes_out = make_layout(p).total;
  return MEGA_MOE_OK;
}

MM_EXPORT int mega_moe_workspace_views(const mega_moe_problem* p, const void* workspace,
                                       mega_moe_views* out) {
  const int st = check_problem(p);
  if (st) return st;
  if (!workspace || !out) return MEGA_MOE_ERR_NULL_POINTER;
  const Layout L = make_layout(p);
  const uint8_t* b = static_cast<const uint8_t*>(workspace);
  out->expert_count = reinterpret_cast<const int32_t*>(b + L.count);
  out->expert_offset = reinterpret_cast<const int32_t*>(b + L.offset);
  out->pool_src = reinterpret_cast<const int32_t*>(b + L.pool_src);
  out->pair_pos = reinterpret_cast<const int32_t*>(b + L.pair_pos);
  out->num_invalid = reinterpret_cast<const int32_t*>(b + L.hdr) + mm::kHdrInvalid;
  out->inter_q = b + L.inter_q;
  out->inter_sf = b + L.inter_sf;
  out->slot = reinterpret_cast<const uint16_t*>(b + L.slot);
  return MEGA_MOE_OK;
}

namespace {
int forward_impl(const mega_moe_problem* p, const void* x, const void* x_sf,
                 const int32_t* topk_idx, const float* topk_w, const void* l1_w,
                 const void* l1_sf, const void* l2_w, const void* l2_sf, void* y,
                 void* workspace, size_t workspace_bytes, void* stream, void* const* events,
                 int num_events, int32_t* recv_stats) {
  int st = check_problem(p);
  if (st) return st;
  const Layout L = make_layout(p);
  if (p->num_tokens == 0) return MEGA_MOE_OK;
  const void* ptrs[] = {x, x_sf, topk_idx, topk_w, l1_w, l1_sf, l2_w, l2_sf, y, workspace};
  for (const void* q : ptrs)
    if (!q) return MEGA_MOE_ERR_NULL_POINTER;
  for (const void* q : ptrs)
    if (misaligned(q)) return MEGA_MOE_ERR_MISALIGNED;
  if (workspace_bytes < L.total) return MEGA_MOE_ERR_WORKSPACE_TOO_SMALL;
  st = check_device();
  if (st) return st;

  mm::Args a{};
  a.x = static_cast<const uint8_t*>(x);
  a.x_sf = x_sf;
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.l1_w = static_cast<const uint8_t*>(l1_w);
  a.l1_sf = l1_sf;
  a.l2_w = static_cast<const uint8_t*>(l2_w);
  a.l2_sf = l2_sf;
  a.y = static_cast<uint16_t*>(y);
  a.recv_stats = recv_stats;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.hdr = reinterpret_cast<int32_t*>(w + L.hdr);
  a.count = reinterpret_cast<int32_t*>(w + L.count);
  a.offset = reinterpret_cast<int32_t*>(w + L.offset);
  a.blk = reinterpret_cast<int32_t*>(w + L.blk);
  a.blk_inv = reinterpret_cast<int32_t*>(w + L.blk_inv);
  a.pair_pos = reinterpret_cast<int32_t*>(w + L.pair_pos);
  a.pool_src = reinterpret_cast<int32_t*>(w + L.pool_src);
  a.w_pool = reinterpret_cast<float*>(w + L.w_pool);
  a.tiles_s = reinterpret_cast<int2*>(w + L.tiles_s);
  a.tiles_l = reinterpret_cast<int2*>(w + L.tiles_l);
  a.x_sf_pool = w + L.x_sf_pool;
  a.inter_q = w + L.inter_q;
  a.inter_sf = w + L.inter_sf;
  a.slot = reinterpret_cast<uint16_t*>(w + L.slot);
  a.tile_done = reinterpret_cast<int32_t*>(w + L.tile_done);
  a.T = (int)p->num_tokens;
  a.H = p->hidden;
  a.I = p->intermediate;
  a.E = p->num_experts;
  a.k = p->topk;
  a.P = L.P;
  a.NB = L.NB;
  a.recipe = p->recipe;
  a.clamp = std::isinf(p->swiglu_clamp) ? 0.f : p->swiglu_clamp;
  a.clamp_inputs = (p->flags & MEGA_MOE_FLAG_CLAMP_INPUTS) != 0;
  a.precise_silu = (p->flags & MEGA_MOE_FLAG_PRECISE_SILU) != 0;
  a.wsf_kmajor = (p->flags & MEGA_MOE_FLAG_WEIGHT_SF_KMAJOR) != 0;
  a.w_paired = (p->flags & MEGA_MOE_FLAG_WEIGHT_E2M1_PAIRED) != 0;
  a.inter64 = (p->flags & MEGA_MOE_FLAG_INTER_SF64) != 0;
  a.tile_mode = (int)(p->flags & MEGA_MOE_FLAG_TILE_MASK);
  a.large_min_rows = mm::kLargeMinRows;
  a.max_tiles_s = L.max_tiles_s;
  a.max_tiles_l = L.max_tiles_l;
  // the large-M kernels address activations, the intermediate and the pool-order scale words
  // through 32-bit buffer descriptors and offsets: larger problems go to the small-M kernels
  if (!mm::large_kernels_addressable(a.T, a.H, a.I, a.k)) a.tile_mode = 1;
  const int cus = device_cus();
  if (cus <= 0) return MEGA_MOE_ERR_HIP;
  a.large_grid = cus < 8 ? 8 : cus / 8 * 8;
  const bool fused = (p->flags & MEGA_MOE_FLAG_FUSED) != 0;
  // the fused forward needs every expert in the large-M class, which needs 32-bit offsets
  if (fused && a.tile_mode == 1) return MEGA_MOE_ERR_INVALID_ARG;
  a.quad = a.recipe == MEGA_MOE_RECIPE_MXFP4W_B32 && a.tile_mode == 0 && !fused;
  a.quad_grid = 2 * a.large_grid;

  hipStream_t s = static_cast<hipStream_t>(stream);
  auto mark = [&](int i) -> bool {
    return i >= num_events || hipEventRecord(static_cast<hipEvent_t>(events[i]), s) == hipSuccess;
  };
  if (!mark(0)) return MEGA_MOE_ERR_HIP;
  if (fused) {   // one launch: every phase event after it
    if (mm::launch_fused(a, s) != hipSuccess) return MEGA_MOE_ERR_HIP;
    for (int i = 1; i < MEGA_MOE_NUM_PHASE_EVENTS; ++i)
      if (!mark(i)) return MEGA_MOE_ERR_HIP;
    return MEGA_MOE_OK;
  }
  if (mm::launch_route(a, s) != hipSuccess || !mark(1)) return MEGA_MOE_ERR_HIP;
  if (mm::launch_l1_small(a, s) != hipSuccess || mm::launch_l1_large(a, s) != hipSuccess || !mark(2))
    return MEGA_MOE_ERR_HIP;
  if (mm::launch_l2_small(a, s) != hipSuccess || mm::launch_l2_large(a, s) != hipSuccess || !mark(3))
    return MEGA_MOE_ERR_HIP;
  if (mm::launch_combine(a, s) != hipSuccess || !mark(4)) return MEGA_MOE_ERR_HIP;
  return MEGA_MOE_OK;
}
}  // namespace

MM_EXPORT int mega_moe_forward(const mega_moe_problem* p, const void* x, const void* x_sf,
                               const int32_t* topk_idx, const float* topk_w, const void* l1_w,
                               const void* l1_sf, const void* l2_w, const void* l2_sf, void* y,
                               void* workspace, size_t workspace_bytes, void* stream) {
  return forward_impl(p, x, x_sf, topk_idx, topk_w, l1_w, l1_sf, l2_w, l2_sf, y, workspace,
                      workspace_bytes, stream, nullptr, 0, nullptr);
}

// ----------------------------------------------------------------------------- no-alloc forward
// The workspace of mega_moe_forward_noalloc: a static device array, one copy per GPU, held until
// the process ends.  In host code `scratch` names a host-side stand-in, not device memory: its
// device address is looked up once per device (hipGetSymbolAddress, with that device current)
// and only that address is ever passed to the kernels.
static __device__ __align__(256) uint8_t scratch[MEGA_MOE_NOALLOC_SCRATCH_BYTES];

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];   // device address of `scratch` on each device (null: not looked up)

// The current device's scratch address, or null when the lookup fails.
void* device_scratch() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* ptr = nullptr;
    if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess || !ptr) return nullptr;
    g_scratch_ptr[dev] = ptr;
  }
  return g_scratch_ptr[dev];
}
}  // namespace

MM_EXPORT int mega_moe_forward_noalloc(const mega_moe_problem* p, const void* x, const void* x_sf,
                                       const int32_t* topk_idx, const float* topk_w, const void* l1_w,
                                       const void* l1_sf, const void* l2_w, const void* l2_sf, void* y,
                                       void* stream) {
  int st = check_problem(p);
  if (st) return st;
  if (p->num_tokens == 0) return MEGA_MOE_OK;
  if (make_layout(p).total > (size_t)MEGA_MOE_NOALLOC_SCRATCH_BYTES) return MEGA_MOE_ERR_SCRATCH_TOO_SMALL;
  st = check_device();
  if (st) return st;
  void* ws = device_scratch();
  if (!ws) return MEGA_MOE_ERR_HIP;
  return forward_impl(p, x, x_sf, topk_idx, topk_w, l1_w, l1_sf, l2_w, l2_sf, y, ws,
                      (size_t)MEGA_MOE_NOALLOC_SCRATCH_BYTES, stream, nullptr, 0, nullptr);
}

MM_EXPORT int mega_moe_forward_stats(const mega_moe_problem* p, const void* x, const void* x_sf,
                                     const int32_t* topk_idx, const float* topk_w, const void* l1_w,
                                     const void* l1_sf, const void* l2_w, const void* l2_sf, void* y,
                                     void* workspace, size_t workspace_bytes,
                                     int32_t* cumulative_expert_recv_stats, void* stream) {
  if ((reinterpret_cast<uintptr_t>(cumulative_expert_recv_stats) & 3u) != 0) return MEGA_MOE_ERR_MISALIGNED;
  return forward_impl(p, x, x_sf, topk_idx, topk_w, l1_w, l1_sf, l2_w, l2_sf, y, workspace,
                      workspace_bytes, stream, nullptr, 0, cumulative_expert_recv_stats);
}

MM_EXPORT int mega_moe_forward_profiled(const mega_moe_problem* p, const void* x, const void* x_sf,
                                        const int32_t* topk_idx, const float* topk_w,
                                        const void* l1_w, const void* l1_sf, const void* l2_w,
                                        const void* l2_sf, void* y, void* workspace,
                                        size_t workspace_bytes, void* stream, void* const* events,
                                        int num_events) {
  if (num_events < 0 || num_events > MEGA_MOE_NUM_PHASE_EVENTS || (num_events > 0 && !events))
    return MEGA_MOE_ERR_INVALID_ARG;
  for (int i = 0; i < num_events; ++i)
    if (!events[i]) return MEGA_MOE_ERR_NULL_POINTER;
  return forward_impl(p, x, x_sf, topk_idx, topk_w, l1_w, l1_sf, l2_w, l2_sf, y, workspace,
                      workspace_bytes, stream, events, num_events, nullptr);
}

MM_EXPORT int mega_moe_transform_weight_scales(const mega_moe_problem* p, const void* l1_sf, const void* l2_sf,
                                               void* l1_sf_kmajor, void* l2_sf_kmajor, void* stream) {
  int st = check_problem(p);
  if (st) return st;
  if (p->recipe == MEGA_MOE_RECIPE_FP8_B128) return MEGA_MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {l1_sf, l2_sf, l1_sf_kmajor, l2_sf_kmajor};
  for (const void* q : ptrs)
    if (!q) return MEGA_MOE_ERR_NULL_POINTER;
  for (const void* q : ptrs)
    if (misaligned(q)) return MEGA_MOE_ERR_MISALIGNED;
  const int H = p->hidden, I = p->intermediate, E = p->num_experts;
  // out of place only: neither output may overlap an input or the other output
  const auto overlap = [](const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
  };
  const size_t n1 = (size_t)E * 2 * I * (H / 32), n2 = (size_t)E * H * (I / 32);
  if (overlap(l1_sf_kmajor, n1, l1_sf, n1) || overlap(l1_sf_kmajor, n1, l2_sf, n2) ||
      overlap(l2_sf_kmajor, n2, l1_sf, n1) || overlap(l2_sf_kmajor, n2, l2_sf, n2) ||
      overlap(l1_sf_kmajor, n1, l2_sf_kmajor, n2))
    return MEGA_MOE_ERR_INVALID_ARG;
  st = check_device();
  if (st) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (mm::launch_sf_kmajor(static_cast<const uint32_t*>(l1_sf), static_cast<uint32_t*>(l1_sf_kmajor), E, 2 * I,
                           H / 128, s) != hipSuccess ||
      mm::launch_sf_kmajor(static_cast<const uint32_t*>(l2_sf), static_cast<uint32_t*>(l2_sf_kmajor), E, H,
                           I / 128, s) != hipSuccess)
    return MEGA_MOE_ERR_HIP;
  return MEGA_MOE_OK;
}

MM_EXPORT int mega_moe_transform_weights(const mega_moe_problem* p, const void* l1_w, const void* l2_w,
                                         void* l1_w_paired, void* l2_w_paired, void* stream) {
  int st = check_problem(p);
  if (st) return st;
  if (p->recipe != MEGA_MOE_RECIPE_MXFP4W_B32) return MEGA_MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {l1_w, l2_w, l1_w_paired, l2_w_paired};
  for (const void* q : ptrs)
    if (!q) return MEGA_MOE_ERR_NULL_POINTER;
  for (const void* q : ptrs)
    if (misaligned(q)) return MEGA_MOE_ERR_MISALIGNED;
  const int H = p->hidden, I = p->intermediate, E = p->num_experts;
  const auto overlap = [](const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
  };
  const size_t n1 = (size_t)E * 2 * I * (H / 2), n2 = (size_t)E * H * (I / 2);
  if (overlap(l1_w_paired, n1, l1_w, n1) || overlap(l1_w_paired, n1, l2_w, n2) ||
      overlap(l2_w_paired, n2, l1_w, n1) || overlap(l2_w_paired, n2, l2_w, n2) ||
      overlap(l1_w_paired, n1, l2_w_paired, n2))
    return MEGA_MOE_ERR_INVALID_ARG;
  st = check_device();
  if (st) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (mm::launch_e2m1_pairs(static_cast<const uint8_t*>(l1_w), static_cast<uint8_t*>(l1_w_paired),
                            (size_t)E * I, H / 128, s) != hipSuccess ||
      mm::launch_e2m1_pairs(static_cast<const uint8_t*>(l2_w), static_cast<uint8_t*>(l2_w_paired),
                            (size_t)E * H / 2, I / 128, s) != hipSuccess)
    return MEGA_MOE_ERR_HIP;
  return MEGA_MOE_OK;
}

MM_EXPORT int mega_moe_diag_mfma_block_sums(int fmt, const void* a, const void* b, const void* a_scale,
                                            const void* b_scale, float* out, int n_tiles, void* stream) {
  if (fmt < 0 || fmt > 2 || n_tiles < 0) return MEGA_MOE_ERR_INVALID_ARG;
  if (n_tiles == 0) return MEGA_MOE_OK;
  if (!a || !b || !out || (fmt != 0 && (!a_scale || !b_scale))) return MEGA_MOE_ERR_NULL_POINTER;
  if (misaligned(a) || misaligned(b) || misaligned(out)) return MEGA_MOE_ERR_MISALIGNED;
  const int st = check_device();
  if (st) return st;
  if (mm::launch_diag_mfma(fmt, static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(b),
                           static_cast<const uint8_t*>(a_scale), static_cast<const uint8_t*>(b_scale), out,
                           n_tiles, static_cast<hipStream_t>(stream)) != hipSuccess)
    return MEGA_MOE_ERR_HIP;
  return MEGA_MOE_OK;
}

// ----------------------------------------------------------- the operators in front of the layer
namespace {

// Byte ranges [lo, hi) of the buffers of one call.
struct Range {
  uintptr_t lo, hi;
};

inline Range range_of(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, p ? a + bytes : a};
}

// Bytes from the first element of the first row to the last element of the last one.
inline size_t rows_bytes(int64_t rows, int64_t stride, int64_t cols, size_t elem) {
  return ((size_t)(rows - 1) * (size_t)stride + (size_t)cols) * elem;
}

inline bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

inline bool known_dtype(int d) { return d == MEGA_MOE_DTYPE_BF16 || d == MEGA_MOE_DTYPE_F32; }
inline size_t dtype_bytes(int d) { return d == MEGA_MOE_DTYPE_BF16 ? 2 : 4; }

constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxTokens = (int64_t)1 << 30;

inline bool bad_stride(int64_t stride, int64_t cols, int64_t step) {
  return stride != 0 && (stride < cols || stride % step || stride >= kMaxStride);
}

inline bool bad_hidden(int h) { return h <= 0 || h % 128 || h > 16384; }

}  // namespace

MM_EXPORT int mega_moe_norm_quant(const mega_moe_norm_problem* p, const void* x, const void* residual,
                                  const void* weight, void* residual_out, void* normed, void* q, void* q_sf,
                                  void* stream) {
  if (!p) return MEGA_MOE_ERR_NULL_POINTER;
  if (p->num_tokens < 0 || p->num_tokens >= kMaxTokens || bad_hidden(p->hidden) || p->flags)
    return MEGA_MOE_ERR_INVALID_ARG;
  if (p->recipe != MEGA_MOE_RECIPE_FP8_B128 && p->recipe != MEGA_MOE_RECIPE_MXFP4W_B32 &&
      p->recipe != MEGA_MOE_RECIPE_MXFP8_B32)
    return MEGA_MOE_ERR_INVALID_ARG;
  if (!known_dtype(p->x_dtype) || !known_dtype(p->weight_dtype)) return MEGA_MOE_ERR_INVALID_ARG;
  if (!(p->eps > 0.f) || std::isinf(p->eps)) return MEGA_MOE_ERR_INVALID_ARG;
  const int64_t T = p->num_tokens, H = p->hidden;
  const size_t xb = dtype_bytes(p->x_dtype);
  if (bad_stride(p->x_stride, H, 16 / (int64_t)xb) || bad_stride(p->residual_stride, H, 16 / (int64_t)xb))
    return MEGA_MOE_ERR_INVALID_ARG;
  if (T == 0) return MEGA_MOE_OK;
  if (!x || !weight || (!q) != (!q_sf)) return MEGA_MOE_ERR_NULL_POINTER;
  if (!normed && !q) return MEGA_MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {x, residual, weight, residual_out, normed, q, q_sf};
  for (const void* ptr : ptrs)
    if (misaligned(ptr)) return MEGA_MOE_ERR_MISALIGNED;
  const int64_t xs = p->x_stride ? p->x_stride : H, rs = p->residual_stride ? p->residual_stride : H;
  const size_t sf_bytes = (size_t)T * (p->recipe == MEGA_MOE_RECIPE_FP8_B128 ? H / 128 * 4 : H / 32);
  const Range in[] = {range_of(x, rows_bytes(T, xs, H, xb)), range_of(residual, rows_bytes(T, rs, H, xb)),
                      range_of(weight, H * dtype_bytes(p->weight_dtype))};
  const Range out[] = {range_of(residual_out, rows_bytes(T, rs, H, xb)), range_of(normed, (size_t)T * H * 2),
                       range_of(q, (size_t)T * H), range_of(q_sf, sf_bytes)};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 3; ++i) {
      // in place: each thread has read its own elements of the row before it writes them
      if (o == 0 && ((i == 1 && residual_out == residual) || (i == 0 && residual_out == x && xs == rs))) continue;
      if (overlap(out[o], in[i])) return MEGA_MOE_ERR_INVALID_ARG;
    }
    for (int k = o + 1; k < 4; ++k)
      if (overlap(out[o], out[k])) return MEGA_MOE_ERR_INVALID_ARG;
  }
  const int st = check_device();
  if (st) return st;
  mm::NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.residual_out = residual_out;
  a.normed = static_cast<uint16_t*>(normed);
  a.q = static_cast<uint8_t*>(q);
  a.q_sf = q_sf;
  a.x_stride = xs;
  a.residual_stride = rs;
  a.T = (int)T;
  a.H = (int)H;
  a.eps = p->eps;
  a.x_f32 = p->x_dtype == MEGA_MOE_DTYPE_F32;
  a.w_f32 = p->weight_dtype == MEGA_MOE_DTYPE_F32;
  a.per32 = p->recipe != MEGA_MOE_RECIPE_FP8_B128;
  return mm::launch_norm_quant(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

MM_EXPORT int mega_moe_gate_logits(const mega_moe_gate_problem* p, const void* x, const void* w, float* logits,
                                   void* stream) {
  if (!p) return MEGA_MOE_ERR_NULL_POINTER;
  if (p->num_tokens < 0 || p->num_tokens >= kMaxTokens || bad_hidden(p->hidden) || p->flags)
    return MEGA_MOE_ERR_INVALID_ARG;
  if (p->num_experts < 1 || p->num_experts > mm::kMaxExperts || !known_dtype(p->weight_dtype) ||
      bad_stride(p->x_stride, p->hidden, 8) || p->x_stride > mm::kMaxGateStride)
    return MEGA_MOE_ERR_INVALID_ARG;
  const int64_t T = p->num_tokens, H = p->hidden, E = p->num_experts;
  if (T == 0) return MEGA_MOE_OK;
  if (!x || !w || !logits) return MEGA_MOE_ERR_NULL_POINTER;
  if (misaligned(x) || misaligned(w) || misaligned(logits)) return MEGA_MOE_ERR_MISALIGNED;
  const int64_t xs = p->x_stride ? p->x_stride : H;
  const Range out = range_of(logits, (size_t)T * E * 4);
  if (overlap(out, range_of(x, rows_bytes(T, xs, H, 2))) ||
      overlap(out, range_of(w, (size_t)E * H * dtype_bytes(p->weight_dtype))))
    return MEGA_MOE_ERR_INVALID_ARG;
  const int st = check_device();
  if (st) return st;
  mm::GateArgs a{};
  a.w = w;
  a.x_stride = xs;
  a.H = (int)H;
  a.E = (int)E;
  a.w_f32 = p->weight_dtype == MEGA_MOE_DTYPE_F32;
  // a launch holds fewer than 2^32 threads: 2^23 tokens of any number of experts
  for (int64_t t = 0; t < T; t += mm::kGateTokens) {
    a.x = static_cast<const uint16_t*>(x) + (size_t)t * xs;
    a.logits = logits + (size_t)t * E;
    a.T = (int)std::min<int64_t>(T - t, mm::kGateTokens);
    if (mm::launch_gate_logits(a, static_cast<hipStream_t>(stream)) != hipSuccess) return MEGA_MOE_ERR_HIP;
  }
  return MEGA_MOE_OK;
}

MM_EXPORT int mega_moe_gate_topk(const mega_moe_topk_problem* p, const void* logits, const float* bias,
                                 const int32_t* num_valid, int32_t* topk_idx, float* topk_w, void* stream) {
  if (!p) return MEGA_MOE_ERR_NULL_POINTER;
  const int64_t T = p->num_tokens, E = p->num_experts, k = p->topk, S = p->num_shared;
  if (T < 0 || E < 1 || S < 0 || E + S > mm::kMaxExperts || k < 1 || k + S > mm::kMaxTopk)
    return MEGA_MOE_ERR_INVALID_ARG;
  if (T >= kMaxTokens || T * (k + S) >= kMaxTokens) return MEGA_MOE_ERR_INVALID_ARG;
  if (p->score != MEGA_MOE_SCORE_SOFTMAX && p->score != MEGA_MOE_SCORE_SIGMOID) return MEGA_MOE_ERR_INVALID_ARG;
  if (!known_dtype(p->logits_dtype) || (p->flags & ~MEGA_MOE_FLAG_TOPK_RENORM)) return MEGA_MOE_ERR_INVALID_ARG;
  const int64_t G = p->num_groups, KG = p->topk_groups;
  if (G < 1 || G > mm::kMaxGroups || E % G || KG < 1 || KG > G || p->group_top < 1 || p->group_top > 2 ||
      k > E / G * KG)
    return MEGA_MOE_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale) || !std::isfinite(p->shared_weight)) return MEGA_MOE_ERR_INVALID_ARG;
  if (bad_stride(p->logits_stride, E, 1)) return MEGA_MOE_ERR_INVALID_ARG;
  if (T == 0) return MEGA_MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MEGA_MOE_ERR_NULL_POINTER;
  if (misaligned(logits) || misaligned(bias) || misaligned(topk_idx) || misaligned(topk_w) ||
      (reinterpret_cast<uintptr_t>(num_valid) & 3u))
    return MEGA_MOE_ERR_MISALIGNED;
  const int64_t ls = p->logits_stride ? p->logits_stride : E;
  const size_t ob = (size_t)T * (k + S) * 4;
  const Range in[] = {range_of(logits, rows_bytes(T, ls, E, dtype_bytes(p->logits_dtype))), range_of(bias, E * 4),
                      range_of(num_valid, 4)};
  const Range oi = range_of(topk_idx, ob), ow = range_of(topk_w, ob);
  if (overlap(oi, ow)) return MEGA_MOE_ERR_INVALID_ARG;
  for (const Range& r : in)
    if (overlap(oi, r) || overlap(ow, r)) return MEGA_MOE_ERR_INVALID_ARG;
  const int st = check_device();
  if (st) return st;
  mm::TopkArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.num_valid = num_valid;
  a.idx = topk_idx;
  a.w = topk_w;
  a.stride = ls;
  a.T = (int)T;
  a.E = (int)E;
  a.k = (int)k;
  a.S = (int)S;
  a.G = (int)G;
  a.KG = (int)KG;
  a.group_top = p->group_top;
  a.sigmoid = p->score == MEGA_MOE_SCORE_SIGMOID;
  a.renorm = (p->flags & MEGA_MOE_FLAG_TOPK_RENORM) != 0;
  a.bf16 = p->logits_dtype == MEGA_MOE_DTYPE_BF16;
  a.scale = p->scale;
  a.shared_weight = p->shared_weight;
  return mm::launch_gate_topk(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

// ------------------------------------------------------------------------------- the layer in parts
namespace {

inline bool known_recipe(int r) {
  return r == MEGA_MOE_RECIPE_FP8_B128 || r == MEGA_MOE_RECIPE_MXFP4W_B32 || r == MEGA_MOE_RECIPE_MXFP8_B32;
}

// Bytes of the scales of `rows` 8-bit rows.
inline size_t scale_bytes(int recipe, int64_t rows, int64_t cols) {
  return (size_t)rows * (recipe == MEGA_MOE_RECIPE_FP8_B128 ? cols / 128 * 4 : cols / 32);
}

// No output overlaps an input or another output.
template <size_t I, size_t O>
bool any_overlap(const Range (&in)[I], const Range (&out)[O]) {
  for (size_t o = 0; o < O; ++o) {
    for (const Range& r : in)
      if (overlap(out[o], r)) return true;
    for (size_t k = o + 1; k < O; ++k)
      if (overlap(out[o], out[k])) return true;
  }
  return false;
}

int check_sort(const mega_moe_sort_problem* p) {
  if (!p) return MEGA_MOE_ERR_NULL_POINTER;
  if (p->num_tokens < 0 || p->num_tokens >= kMaxTokens || bad_hidden(p->hidden) || p->flags || p->num_experts < 1 ||
      p->num_experts > mm::kMaxExperts || p->topk < 1 || p->topk > mm::kMaxTopk || !known_recipe(p->recipe))
    return MEGA_MOE_ERR_INVALID_ARG;
  if (p->num_tokens * p->topk >= kMaxTokens) return MEGA_MOE_ERR_INVALID_ARG;
  if (!known_dtype(p->dtype) && p->dtype != MEGA_MOE_DTYPE_E4M3) return MEGA_MOE_ERR_INVALID_ARG;
  const int64_t step = p->dtype == MEGA_MOE_DTYPE_E4M3 ? 16 : 16 / (int64_t)dtype_bytes(p->dtype);
  return bad_stride(p->x_stride, p->hidden, step) ? MEGA_MOE_ERR_INVALID_ARG : MEGA_MOE_OK;
}

// The workspace: block counts, then the experts' totals.
size_t sort_workspace(const mega_moe_sort_problem* p) {
  const int64_t P = p->num_tokens * p->topk;
  if (P <= mm::kSortSmallPairs) return 0;
  return align256((size_t)mm::sort_blocks(P) * p->num_experts * 4) + align256((size_t)p->num_experts * 4);
}

int check_unsort(const mega_moe_unsort_problem* p) {
  if (!p) return MEGA_MOE_ERR_NULL_POINTER;
  if (p->num_tokens < 0 || p->num_tokens >= kMaxTokens || p->num_rows < 0 || p->num_rows > kMaxTokens ||
      bad_hidden(p->hidden) || p->flags || p->topk < 1 || p->topk > mm::kMaxTopk || !known_dtype(p->dtype))
    return MEGA_MOE_ERR_INVALID_ARG;
  if (p->num_tokens * p->topk >= kMaxTokens) return MEGA_MOE_ERR_INVALID_ARG;
  return bad_stride(p->stride, p->hidden, 16 / (int64_t)dtype_bytes(p->dtype)) ? MEGA_MOE_ERR_INVALID_ARG : MEGA_MOE_OK;
}

mm::UnsortArgs unsort_args(const mega_moe_unsort_problem* p) {
  mm::UnsortArgs a{};
  a.T = (int)p->num_tokens;
  a.H = p->hidden;
  a.k = p->topk;
  a.R = (int)(p->num_rows ? p->num_rows : p->num_tokens * p->topk);
  a.f32 = p->dtype == MEGA_MOE_DTYPE_F32;
  a.stride = p->stride ? p->stride : p->hidden;
  return a;
}

int check_act(const mega_moe_act_problem* p) {
  if (!p) return MEGA_MOE_ERR_NULL_POINTER;
  if (p->num_rows < 0 || p->num_rows >= kMaxTokens || bad_hidden(p->width) || !known_recipe(p->recipe) ||
      !known_dtype(p->x_dtype) || (p->act != MEGA_MOE_ACT_NONE && p->act != MEGA_MOE_ACT_SWIGLU) ||
      (p->flags & ~MEGA_MOE_FLAG_CLAMP_INPUTS) || std::isnan(p->swiglu_clamp) || p->swiglu_clamp < 0.f)
    return MEGA_MOE_ERR_INVALID_ARG;
  if (p->act == MEGA_MOE_ACT_NONE && (p->flags || p->swiglu_clamp != 0.f)) return MEGA_MOE_ERR_INVALID_ARG;
  const int64_t cols = p->act == MEGA_MOE_ACT_SWIGLU ? 2 * (int64_t)p->width : p->width;
  return bad_stride(p->x_stride, cols, 16 / (int64_t)dtype_bytes(p->x_dtype)) ? MEGA_MOE_ERR_INVALID_ARG : MEGA_MOE_OK;
}

mm::ActArgs act_args(const mega_moe_act_problem* p) {
  mm::ActArgs a{};
  a.M = (int)p->num_rows;
  a.I = p->width;
  a.swiglu = p->act == MEGA_MOE_ACT_SWIGLU;
  a.x_stride = p->x_stride ? p->x_stride : (a.swiglu ? 2 * (int64_t)p->width : p->width);
  a.clamp = std::isinf(p->swiglu_clamp) ? 0.f : p->swiglu_clamp;
  a.clamp_inputs = (p->flags & MEGA_MOE_FLAG_CLAMP_INPUTS) != 0;
  a.f32 = p->x_dtype == MEGA_MOE_DTYPE_F32;
  a.per32 = p->recipe != MEGA_MOE_RECIPE_FP8_B128;
  return a;
}

inline bool misaligned4(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 3u) != 0; }

}  // namespace

MM_EXPORT int mega_moe_sort_workspace_size(const mega_moe_sort_problem* p, size_t* bytes_out) {
  const int st = check_sort(p);
  if (st) return st;
  if (!bytes_out) return MEGA_MOE_ERR_NULL_POINTER;
  *bytes_out = sort_workspace(p);
  return MEGA_MOE_OK;
}

MM_EXPORT int mega_moe_sort_tokens(const mega_moe_sort_problem* p, const void* x, const void* x_sf,
                                   const int32_t* topk_idx, void* rows, void* rows_sf, int32_t* pool_src,
                                   int32_t* pair_pos, int32_t* expert_offset, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  const int bad = check_sort(p);
  if (bad) return bad;
  const int64_t T = p->num_tokens, H = p->hidden, E = p->num_experts, P = T * p->topk;
  const bool bytes8 = p->dtype == MEGA_MOE_DTYPE_E4M3;
  const size_t elem = bytes8 ? 1 : dtype_bytes(p->dtype);
  if (!expert_offset) return MEGA_MOE_ERR_NULL_POINTER;
  if (misaligned(expert_offset)) return MEGA_MOE_ERR_MISALIGNED;
  mm::SortArgs a{};
  a.offset = expert_offset;
  a.E = (int)E;
  if (T > 0) {
    if (!topk_idx || !pool_src || !pair_pos || (!x) != (!rows)) return MEGA_MOE_ERR_NULL_POINTER;
    if (x && bytes8 && (!x_sf || !rows_sf)) return MEGA_MOE_ERR_NULL_POINTER;
    if ((!x || !bytes8) && (x_sf || rows_sf)) return MEGA_MOE_ERR_INVALID_ARG;
    const void* ptrs[] = {x, x_sf, topk_idx, rows, rows_sf, pool_src, pair_pos, workspace};
    for (const void* ptr : ptrs)
      if (misaligned(ptr)) return MEGA_MOE_ERR_MISALIGNED;
    const size_t need = sort_workspace(p);
    if (need && (!workspace || workspace_bytes < need)) return MEGA_MOE_ERR_WORKSPACE_TOO_SMALL;
    const int64_t xs = p->x_stride ? p->x_stride : H;
    const Range in[] = {range_of(x, rows_bytes(T, xs, H, elem)), range_of(x_sf, scale_bytes(p->recipe, T, H)),
                        range_of(topk_idx, (size_t)P * 4)};
    const Range out[] = {range_of(rows, (size_t)P * H * elem), range_of(rows_sf, scale_bytes(p->recipe, P, H)),
                         range_of(pool_src, (size_t)P * 4), range_of(pair_pos, (size_t)P * 4),
                         range_of(expert_offset, (size_t)(E + 1) * 4), range_of(need ? workspace : nullptr, need)};
    if (any_overlap(in, out)) return MEGA_MOE_ERR_INVALID_ARG;
    a.x = x;
    a.x_sf = static_cast<const uint32_t*>(x_sf);
    a.idx = topk_idx;
    a.rows = rows;
    a.rows_sf = static_cast<uint32_t*>(rows_sf);
    a.src = pool_src;
    a.pos = pair_pos;
    a.x_stride = (size_t)xs * elem;
    a.T = (int)T;
    a.k = p->topk;
    a.P = (int)P;
    a.row_bytes = (int)(H * elem);
    a.sf_words = (int)(H / 128);               // a float, or four codes, for each 128 columns
    if (need) {
      a.NB = mm::sort_blocks(P);
      a.block_pairs = mm::sort_block_pairs(P);
      a.blk = static_cast<int32_t*>(workspace);
      a.total = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + align256((size_t)a.NB * E * 4));
    }
  }
  const int st = check_device();
  if (st) return st;
  return mm::launch_sort(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

MM_EXPORT int mega_moe_unsort_tokens(const mega_moe_unsort_problem* p, const void* rows, const int32_t* pair_pos,
                                     const float* topk_w, void* y, void* stream) {
  const int bad = check_unsort(p);
  if (bad) return bad;
  if (p->num_tokens == 0) return MEGA_MOE_OK;
  if (!rows || !pair_pos || !y) return MEGA_MOE_ERR_NULL_POINTER;
  if (misaligned(rows) || misaligned(pair_pos) || misaligned(topk_w) || misaligned(y)) return MEGA_MOE_ERR_MISALIGNED;
  mm::UnsortArgs a = unsort_args(p);
  const size_t elem = dtype_bytes(p->dtype), pairs = (size_t)a.T * a.k * 4;
  const Range in[] = {range_of(rows, (size_t)a.R * a.H * elem), range_of(pair_pos, pairs), range_of(topk_w, pairs)};
  const Range out[] = {range_of(y, rows_bytes(a.T, a.stride, a.H, elem))};
  if (any_overlap(in, out)) return MEGA_MOE_ERR_INVALID_ARG;
  const int st = check_device();
  if (st) return st;
  a.rows = rows;
  a.pos = pair_pos;
  a.w = topk_w;
  a.y = y;
  return mm::launch_unsort(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

MM_EXPORT int mega_moe_unsort_backward(const mega_moe_unsort_problem* p, const void* dy, const void* rows,
                                       const int32_t* pair_pos, const float* topk_w, void* d_rows, float* d_w,
                                       void* stream) {
  const int bad = check_unsort(p);
  if (bad) return bad;
  if (p->num_tokens == 0) return MEGA_MOE_OK;
  if (!dy || !pair_pos || (d_w && !rows)) return MEGA_MOE_ERR_NULL_POINTER;
  if (!d_rows && !d_w) return MEGA_MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {dy, rows, pair_pos, topk_w, d_rows, d_w};
  for (const void* ptr : ptrs)
    if (misaligned(ptr)) return MEGA_MOE_ERR_MISALIGNED;
  mm::UnsortArgs a = unsort_args(p);
  const size_t elem = dtype_bytes(p->dtype), pairs = (size_t)a.T * a.k * 4, all = (size_t)a.R * a.H * elem;
  // in place: each thread has read its own columns of a pair's row before it writes them
  const Range in[] = {range_of(dy, rows_bytes(a.T, a.stride, a.H, elem)), range_of(d_rows == rows ? nullptr : rows, all),
                      range_of(pair_pos, pairs), range_of(topk_w, pairs)};
  const Range out[] = {range_of(d_rows, all), range_of(d_w, pairs)};
  if (any_overlap(in, out)) return MEGA_MOE_ERR_INVALID_ARG;
  const int st = check_device();
  if (st) return st;
  a.dy = dy;
  a.rows = rows;
  a.pos = pair_pos;
  a.w = topk_w;
  a.d_rows = d_rows;
  a.d_w = d_w;
  return mm::launch_unsort_backward(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

MM_EXPORT int mega_moe_block_product(const mega_moe_product_problem* p, const void* x, const float* x_sf, const void* w,
                                     const float* w_sf, const int32_t* group_offset, void* y, void* stream) {
  if (!p) return MEGA_MOE_ERR_NULL_POINTER;
  if (p->num_rows < 0 || p->num_rows >= kMaxTokens || p->n <= 0 || p->n % 8 || p->n > mm::kMaxProductN || bad_hidden(p->k) ||
      p->num_groups < 1 || p->num_groups > mm::kMaxExperts || p->flags || bad_stride(p->x_stride, p->k, 16) ||
      p->x_stride > mm::kMaxProductStride || bad_stride(p->y_stride, p->n, 8) ||
      p->num_rows * p->n >= mm::kMaxProductArea)
    return MEGA_MOE_ERR_INVALID_ARG;
  const int64_t M = p->num_rows, N = p->n, K = p->k, G = p->num_groups;
  if (M == 0) return MEGA_MOE_OK;
  if (!x || !x_sf || !w || !w_sf || !y || (G > 1 && !group_offset)) return MEGA_MOE_ERR_NULL_POINTER;
  if (misaligned(x) || misaligned(x_sf) || misaligned(w) || misaligned(w_sf) || misaligned(y) || misaligned4(group_offset))
    return MEGA_MOE_ERR_MISALIGNED;
  const int64_t xs = p->x_stride ? p->x_stride : K, ys = p->y_stride ? p->y_stride : N;
  const Range in[] = {range_of(x, rows_bytes(M, xs, K, 1)), range_of(x_sf, (size_t)M * (K / 128) * 4),
                      range_of(w, (size_t)G * N * K), range_of(w_sf, (size_t)G * ((N + 127) / 128) * (K / 128) * 4),
                      range_of(group_offset, (size_t)(G + 1) * 4)};
  const Range out[] = {range_of(y, rows_bytes(M, ys, N, 2))};
  if (any_overlap(in, out)) return MEGA_MOE_ERR_INVALID_ARG;
  const int st = check_device();
  if (st) return st;
  mm::ProductArgs a{};
  a.x = static_cast<const uint8_t*>(x);
  a.x_sf = x_sf;
  a.w = static_cast<const uint8_t*>(w);
  a.w_sf = w_sf;
  a.offset = group_offset;
  a.y = static_cast<uint16_t*>(y);
  a.x_stride = xs;
  a.y_stride = ys;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.G = (int)G;
  return mm::launch_product(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

MM_EXPORT int mega_moe_act_quant(const mega_moe_act_problem* p, const void* x, const int32_t* num_valid, void* q,
                                 void* q_sf, void* out, void* stream) {
  const int bad = check_act(p);
  if (bad) return bad;
  if (p->num_rows == 0) return MEGA_MOE_OK;
  if (!x || (!q) != (!q_sf)) return MEGA_MOE_ERR_NULL_POINTER;
  if (!q && !out) return MEGA_MOE_ERR_INVALID_ARG;
  if (misaligned(x) || misaligned(q) || misaligned(q_sf) || misaligned(out) || misaligned4(num_valid))
    return MEGA_MOE_ERR_MISALIGNED;
  mm::ActArgs a = act_args(p);
  const int64_t M = a.M, I = a.I;
  const Range in[] = {range_of(x, rows_bytes(M, a.x_stride, a.swiglu ? 2 * I : I, dtype_bytes(p->x_dtype))),
                      range_of(num_valid, 4)};
  const Range outs[] = {range_of(q, (size_t)M * I), range_of(q_sf, scale_bytes(p->recipe, M, I)),
                        range_of(out, (size_t)M * I * 2)};
  if (any_overlap(in, outs)) return MEGA_MOE_ERR_INVALID_ARG;
  const int st = check_device();
  if (st) return st;
  a.x = x;
  a.num_valid = num_valid;
  a.q = static_cast<uint8_t*>(q);
  a.q_sf = q_sf;
  a.out = static_cast<uint16_t*>(out);
  return mm::launch_act_quant(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

MM_EXPORT int mega_moe_act_backward(const mega_moe_act_problem* p, const void* x, const void* d_out,
                                    const int32_t* num_valid, void* d_x, void* stream) {
  const int bad = check_act(p);
  if (bad) return bad;
  if (p->act != MEGA_MOE_ACT_SWIGLU) return MEGA_MOE_ERR_INVALID_ARG;
  if (p->num_rows == 0) return MEGA_MOE_OK;
  if (!x || !d_out || !d_x) return MEGA_MOE_ERR_NULL_POINTER;
  if (misaligned(x) || misaligned(d_out) || misaligned(d_x) || misaligned4(num_valid)) return MEGA_MOE_ERR_MISALIGNED;
  mm::ActArgs a = act_args(p);
  const size_t elem = dtype_bytes(p->x_dtype), wide = rows_bytes(a.M, a.x_stride, 2 * (int64_t)a.I, elem);
  // in place: each thread has read its own columns before it writes them
  const Range in[] = {range_of(d_x == x ? nullptr : x, wide), range_of(d_out, (size_t)a.M * a.I * elem),
                      range_of(num_valid, 4)};
  const Range out[] = {range_of(d_x, wide)};
  if (any_overlap(in, out)) return MEGA_MOE_ERR_INVALID_ARG;
  const int st = check_device();
  if (st) return st;
  a.x = x;
  a.num_valid = num_valid;
  a.d_out = d_out;
  a.d_x = d_x;
  return mm::launch_act_backward(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}
