// 8-bit matrix product with a scale for each block of 128, by group of rows or dense:
//
//   y[m, n] = bf16( sum_b sx[m, b] sw[g, n / 128, b] sum_{k in b} x[m, k] w[g, n, k] )
//
// Weight rows are the MFMA's A operand and x's rows its B operand, so a lane ends with four consecutive columns of one
// row of y.  A 16x16x128 MFMA spans one block; its result is scaled and added to the float32 sums: four multiply-adds a lane
// and MFMA, half of the vector unit's time while the matrix unit is busy.
#include "mm_parts.h"
#include "mm_product_policy.h"
#include "mm_route_dev.h"
#include "mm_rows.h"

namespace mm {
namespace {

// One block of 128: the instruction without block scales (scale operands 0).
__device__ __forceinline__ v4f mfma_block(const v8i& a, const v8i& b) {
  const v4f z = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
}

// A launch's part of the items: slabs of weight rows times tiles of rows, `count` of them from `first`.
struct ProductPart {
  int slabs, tiles, first, count;
};

// ------------------------------------------------------------------------------- many rows
// A workgroup takes 64 kWN weight rows x 16 kNG kWM rows of x, its eight waves (two a SIMD) 64 weight rows (wm = wave % kWN)
// and kNG groups of 16 rows of x (kWM i + wave / kWN) each.  With kKS 2 the waves are two sets of four that take every other
// block, and the second set's sums are added to the first's at the end: half the barriers, for one step more to fill and the
// hand-over (128 x 64 tiles, us, kKS 1 and 2: 512 x 4096 x 7168 28.1, 25.0; 777 x 2120 x 3712 15.0, 15.5; 2048 x 512 x 512 4.8, 5.1).
// Blocks of 128 columns of both operands, with the rows' scales, go through a
// ring in LDS by loads that need no registers; a block's MFMAs run while the next ones are on their way.  16-byte chunk c of
// a row r sits at c ^ (r / 2 % 8), so that the 16 rows of an operand read fall into different banks.
//
// 8192 x 4096 x 7168 in tiles of 256 x 256 takes 218 to 231 us by box, 2080 to 2210 TFLOP/s, of the 160 us at the 3000 TFLOP/s
// that a large library product with one scale a tensor reaches here.  The matrix units are busy half of the cycles (2.1 GHz on
// the loaded chip): a block takes about 4100 for 2048 of MFMAs.  The scaling (four multiply-adds an MFMA) runs beside the MFMAs
// in a register-only loop (4% longer than without), LDS is busy a quarter of the time, and with every workgroup on the same
// tile, so that all lines come from the L2, it still takes 204 us; the loop without barriers or without loads has not been
// timed, so the rest is not explained.  (Times of a change, here and below, are of one box each.)  Three blocks of 256 x 256 do
// not fit into LDS; 256 x 128 with three takes 241.  32x32x64 MFMAs save nothing (256 x 128: 255 us against 246) and spill at
// 256 x 256.  Loads in one burst behind the first group's MFMAs: 230; band heights 2 and 8 instead of 4: 232, 226.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)(uint32_t)bytes, 0x00020000);
}
__device__ __forceinline__ void lds_load16(rsrc_t r, uint32_t voff, uint32_t soff, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, (int)soff, 0, 0);
}
__device__ __forceinline__ void lds_load4(rsrc_t r, uint32_t voff, uint32_t soff, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 4, voff, (int)soff, 0, 0);
}
template <int kN>
__device__ __forceinline__ void wait_vmcnt() {
  __builtin_amdgcn_s_waitcnt((kN & 0xF) | ((kN >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
// Barrier of the block loop: every wave has waited for its own loads, which are then in LDS.
__device__ __forceinline__ void pipeline_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ v8i lds_operand(const uint8_t* lo, const uint8_t* hi, int off) {
  const v4i a = *reinterpret_cast<const v4i*>(lo + off);
  const v4i b = *reinterpret_cast<const v4i*>(hi + off);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Tile `t` of the tiles of at most kBM rows that the groups are cut into: its group, first row and rows (0: there is none).
template <int kBM, int kThreads>
__device__ __forceinline__ Tile find_tile(const ProductArgs& a, int t, int tiles, uint32_t* sh, Tile* found) {
  if (!a.offset) return Tile{0, t * kBM, min(kBM, a.M - t * kBM)};
  const int tid = threadIdx.x, per = (a.G + kThreads - 1) / kThreads;
  const int g0 = min(tid * per, a.G), g1 = min(g0 + per, a.G);
  if (tid == 0) *found = Tile{0, 0, 0};
  const uint32_t sum = tiles_of(a.offset, g0, g1, a.M, kBM, tiles);
  uint32_t v[1] = {sum}, all[1];
  block_scan_n<1, kThreads>(v, sh, all);
  const uint32_t before = v[0] - sum;
  if ((uint32_t)t >= before && (uint32_t)t < v[0]) *found = tile_among(a.offset, g0, g1, a.M, kBM, (uint32_t)t - before);
  __syncthreads();
  return *found;
}

template <int kNG, int kWN, int kKS, int kStages>
struct LargeLds {
  static constexpr int kBN = 64 * kWN, kWM = 8 / kWN / kKS, kBM = 16 * kNG * kWM;
  static constexpr int kW = kBN * 128, kX = kBM * 128, kBlock = kW + kX + kBM * 16, kStage = kKS * kBlock;
  uint8_t ring[kStages * kStage];
  float wsc[(kBN + 127) / 128][kMaxKBlocks];
  uint32_t sh[32];
  Tile tile;
};

template <int kNG, int kWN, int kKS, int kStages>
__global__ __launch_bounds__(512) void k_product_large(ProductArgs a, ProductPart part) {
  using L = LargeLds<kNG, kWN, kKS, kStages>;
  constexpr int kBN = L::kBN, kBM = L::kBM, kWM = L::kWM, kGW = 8 / kKS;     // kGW: waves that share a block
  constexpr int kWLoads = kBN / 8 / kGW, kXLoads = (kBM / 8 + kGW - 1) / kGW, kSLoads = (kBM / 16 + kGW - 1) / kGW,
                kLoads = kWLoads + kXLoads + kSLoads;
  constexpr bool kAhead = kNG > 1 && kKS == 1;   // operands of a block's first group are read in the block before
  constexpr int kParts = !kAhead ? 1 : kNG < 4 ? kNG : 4;   // a block's loads go out behind the MFMAs of that many groups of rows
  static_assert((kStages - 1) * kLoads < 64, "vmcnt holds 6 bits");
  __shared__ __align__(1024) L lds;
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const int w8 = __builtin_amdgcn_readfirstlane(tid >> 6), ks = w8 / kGW, w = w8 % kGW, wm = w % kWN, wn = w / kWN;
  const int KB = a.K / 128, steps = (KB + kKS - 1) / kKS;
  // each XCD walks a contiguous range of items; an item is (band of 4 tiles, slab, tile of the band)
  const int at = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3), item = part.first + at;
  if (at >= part.count) return;
  const int slabs = part.slabs, band = item / (4 * slabs), in = item - band * 4 * slabs, high = min(4, part.tiles - 4 * band);
  const int slab = in / high, t = 4 * band + in - slab * high;
  const Tile tile = find_tile<kBM, 512>(a, t, part.tiles, lds.sh, &lds.tile);
  if (tile.rows <= 0) return;
  const int g = __builtin_amdgcn_readfirstlane(tile.g), m0 = __builtin_amdgcn_readfirstlane(tile.m0),
            rows = __builtin_amdgcn_readfirstlane(tile.rows), n0 = slab * kBN, nrows = min(kBN, a.N - n0);

  const rsrc_t wr = make_rsrc(a.w + ((size_t)g * a.N + n0) * a.K, (size_t)nrows * a.K);
  const rsrc_t xr = make_rsrc(a.x + (size_t)m0 * a.x_stride, (size_t)(rows - 1) * a.x_stride + a.K);
  const rsrc_t sr = make_rsrc(a.x_sf + (size_t)m0 * KB, (size_t)rows * KB * 4);
  // LDS row 64 wm + 16 rt + m of the weights holds row 64 wm + 16 (m / 4) + 4 rt + m % 4 of the slab, so that a lane's four
  // tiles are 16 consecutive columns of y.  Rows past the last one lie past the buffer's end and read zeros; rows of x past
  // the tile's last repeat that one.  Where a wave has no piece of its own left, it fetches the last one again.
  uint32_t wo[kWLoads], xo[kXLoads], so[kSLoads];
#pragma unroll
  for (int j = 0; j < kWLoads; ++j) {
    const int r = 8 * (kWLoads * w + j) + (lane >> 3), m = r & 15;
    const int n = (r & ~63) + 16 * (m >> 2) + 4 * ((r >> 4) & 3) + (m & 3);
    wo[j] = (uint32_t)n * (uint32_t)a.K + 16u * (uint32_t)((lane & 7) ^ ((r >> 1) & 7));
  }
  const auto x_piece = [&](int j) { return min(w + kGW * j, kBM / 8 - 1); };
  const auto s_piece = [&](int j) { return min(w + kGW * j, kBM / 16 - 1); };
#pragma unroll
  for (int j = 0; j < kXLoads; ++j) {
    const int r = 8 * x_piece(j) + (lane >> 3);
    xo[j] = (uint32_t)min(r, rows - 1) * (uint32_t)a.x_stride + 16u * (uint32_t)((lane & 7) ^ ((r >> 1) & 7));
  }
#pragma unroll
  for (int j = 0; j < kSLoads; ++j) {
    const int r = 16 * s_piece(j) + (lane >> 2);
    so[j] = ((uint32_t)min(r, rows - 1) * (uint32_t)KB + (uint32_t)(lane & 3)) * 4u;
  }
  // In the largest tiles the XCDs start at different columns and wrap round, so that they do not all ask for the same columns of
  // their rows at once (8192 x 4096 x 7168 222 -> 217 us, 8192 x 7168 x 2048 140 -> 129; smaller tiles lose up to 5%).
  const int rot = kNG == 8 ? (int)(blockIdx.x & 7) * KB / 8 : 0;
  const auto turned = [&](int kb) { return kNG < 8 || kb + rot < KB ? kb + rot : kb + rot - KB; };
  const auto stage = [&](int slot) { return lds.ring + slot * L::kStage + ks * L::kBlock; };
  // A wave's share of its block of step i.  Loads past the last block count but fetch nothing: a lane offset of 2^31 lies past any
  // buffer's end.
  const auto fetch = [&](int step, int slot, int part, int parts) {
    uint8_t* to = stage(slot);
    const int kb = kKS * step + ks;
    const uint32_t past = kb < KB ? 0u : 0x80000000u, k = kb < KB ? (uint32_t)turned(kb) : 0u;
#pragma unroll
    for (int i = kLoads * part / parts; i < kLoads * (part + 1) / parts; ++i) {
      const int x = i - kWLoads, f = x - kXLoads;
      if (x < 0) lds_load16(wr, wo[i] + past, k * 128, to + (kWLoads * w + i) * 1024);
      else if (f < 0) lds_load16(xr, xo[x] + past, k * 128, to + L::kW + x_piece(x) * 1024);
      else lds_load4(sr, so[f] + past, (k & ~3u) * 4, to + L::kW + L::kX + s_piece(f) * 256);
    }
  };
  {
    const int nb = (a.N + 127) / 128;
    for (int i = tid; i < (kBN + 127) / 128 * KB; i += 512) {
      const int h = i / KB, b = i - h * KB;
      lds.wsc[h][b] = a.w_sf[((size_t)g * nb + min(n0 / 128 + h, nb - 1)) * KB + b];
    }
  }
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(s, s, 0, 1);
  if (kAhead) fetch(kStages - 1, kStages - 1, 0, kParts);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");

  const int sw7 = (lr >> 1) & 7, arow = 64 * wm + lr, xrow = 16 * wn + lr;
  const int alo = arow * 128 + 16 * (lg ^ sw7), ahi = arow * 128 + 16 * ((lg | 4) ^ sw7);
  const int xlo = L::kW + xrow * 128 + 16 * (lg ^ sw7), xhi = L::kW + xrow * 128 + 16 * ((lg | 4) ^ sw7);
  const int slo = L::kW + L::kX + xrow * 16;
  constexpr int kGroup = 16 * kWM * 128;         // bytes from one group of rows of x to the next
  const float* wsc = lds.wsc[wm >> 1];

  v4f acc[4][kNG], pend[4];
  float pend_s = 0.f;
#pragma unroll
  for (int rt = 0; rt < 4; ++rt) {
    pend[rt] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kNG; ++i) acc[rt][i] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  // Where there is more than one group of rows, the operands of a block's first group are read in the block before, behind its
  // last group's MFMAs, and the barrier stands in front of those: it is passed with MFMAs still to issue on either side
  // (8192 x 4096 x 7168 213 -> 209 us).  With one group nothing is left to issue there (777 x 2120 x 3712 16.0, ahead 18.6).
  v8i A[4], B;
  const auto read_first = [&](const uint8_t* S) {
    B = lds_operand(S + xlo, S + xhi, 0);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) A[rt] = lds_operand(S + alo, S + ahi, rt * 2048);
  };
  if (kAhead) {
    wait_vmcnt<(kStages - 2) * kLoads + kLoads / kParts>();
    pipeline_barrier();
    read_first(stage(0));
  }
  int slot = 0;
  for (int step = 0; step < steps; ++step) {
    const int kb = kKS * step + ks, at = turned(kb);
    const uint8_t* S = stage(slot);
    const int last = slot == 0 ? kStages - 1 : slot - 1, next = slot + 1 == kStages ? 0 : slot + 1;
    if (!kAhead) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      wait_vmcnt<(kStages - 2) * kLoads>();
      pipeline_barrier();                        // the block is in LDS, the one before has been read
    }
    if (kKS == 1 || kb < KB) {                   // no wave is left out of a barrier
      v4f p[2][4];
      float sx[kNG];
      if (!kAhead) read_first(S);
      const float cw = wsc[at];
#pragma unroll
      for (int i = 0; i < kNG; ++i) {
        v8i Bn = B;
        if (i + 1 < kNG) Bn = lds_operand(S + xlo, S + xhi, kGroup * (i + 1));
        if (i == 0) {
#pragma unroll
          for (int n = 0; n < kNG; ++n) sx[n] = *reinterpret_cast<const float*>(S + slo + kGroup / 8 * n + 4 * (at & 3));
        }
        if (kAhead && i + 1 == kNG) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // this block has been read
          wait_vmcnt<(kStages - 2) * kLoads>();
          pipeline_barrier();                      // by every wave, and the next one is in LDS
        }
        const float sc = i > 0 ? sx[i - 1] * cw : pend_s;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          p[i & 1][rt] = mfma_block(A[rt], B);
          if (i > 0) acc[rt][i - 1] += p[(i - 1) & 1][rt] * sc;
          else acc[rt][kNG - 1] += pend[rt] * sc;
        }
        if (i + 1 < kNG) {
          __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
          if (i + 1 < kParts) {
            fetch(step + kStages - 1, last, i + 1, kParts);
            __builtin_amdgcn_sched_barrier(0);
          }
          B = Bn;
        } else {
          __builtin_amdgcn_sched_barrier(0);
          if (kAhead) read_first(stage(next));
          __builtin_amdgcn_sched_barrier(0);
          if (kAhead) fetch(step + kStages, slot, 0, kParts);
          else if (kKS == 1) fetch(step + kStages - 1, last, 0, 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) pend[rt] = p[(kNG - 1) & 1][rt];
      pend_s = sx[kNG - 1] * cw;
    }
    if (kKS > 1) fetch(step + kStages - 1, last, 0, 1);
    slot = next;
  }
#pragma unroll
  for (int rt = 0; rt < 4; ++rt) acc[rt][kNG - 1] += pend[rt] * pend_s;
  wait_vmcnt<0>();                               // nothing may land in LDS after the workgroup's end
  if constexpr (kKS > 1) {                       // the waves of the other blocks hand over their sums
    static_assert(kKS == 2 && kGW * 4 * kNG * 1024 <= kStages * L::kStage, "");
    v4f* const sums = reinterpret_cast<v4f*>(lds.ring) + w * 4 * kNG * 64 + lane;
    __syncthreads();
    if (ks == 1) {
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int i = 0; i < kNG; ++i) sums[(rt * kNG + i) * 64] = acc[rt][i];
    }
    __syncthreads();
    if (ks == 1) return;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int i = 0; i < kNG; ++i) acc[rt][i] += sums[(rt * kNG + i) * 64];
  }

  const int n = n0 + 64 * wm + 16 * lg;
#pragma unroll
  for (int i = 0; i < kNG; ++i) {
    const int r = 16 * (kWM * i + wn) + lr;
    if (r >= rows) continue;
    uint16_t* y = a.y + (size_t)(m0 + r) * a.y_stride + n;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (n + 8 * h >= a.N) continue;
      const v4f &u = acc[2 * h][i], &v = acc[2 * h + 1][i];
      *reinterpret_cast<uint4*>(y + 8 * h) =
          make_uint4(pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]), pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
  }
}

// ------------------------------------------------------------------------------- few tiles
// Where there are fewer large tiles than compute units: a workgroup takes 16 kRT weight rows x 16 kCT rows of x, and its kWaves
// waves share K, wave w the blocks w, w + kWaves, ..., each for the whole tile through a ring of kStages blocks of its own in
// LDS, so the loop has no barrier; the waves' sums meet in LDS in a fixed order.  Rows are fetched as whole 128-byte lines, 8
// rows x 128 bytes a load; operands loaded straight into registers touch 64 bytes of 16 rows, half of what the L2 delivers for
// them (1 x 4096 x 7168 in the same tiles 8.7 us instead of 7.0, 128 x 4096 x 7168 30.0 instead of 12.4).  One row of 4096 x 7168
// is bound by the weights' 29 MB, 5.8 us at the rate of a large copy.
template <int kRT, int kCT, int kWaves, int kStages, int kBlocks>
struct SplitLds {
  static constexpr int kX = 2048 * kCT, kBlock = 2048 * kRT + kX, kRing = kStages * kBlock;
  static constexpr int kSums = kWaves * kRT * kCT * 1024, kMain = kWaves * kRing > kSums ? kWaves * kRing : kSums;
  uint8_t main[kMain];                           // the waves' rings, then their sums
  float sw[kMaxKBlocks], sx[16 * kCT * (kBlocks | 1)];   // the weights' scales [KB], the rows' [16 kCT][KB | 1]
  uint32_t sh[32];
  Tile tile;
};

template <int kRT, int kCT, int kWaves, int kStages, int kBlocks>
__global__ __launch_bounds__(64 * kWaves) void k_product_split(ProductArgs a, ProductPart part) {
  using L = SplitLds<kRT, kCT, kWaves, kStages, kBlocks>;
  constexpr int kLoads = 2 * (kRT + kCT);
  __shared__ __align__(1024) L lds;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), lr = lane & 15, lg = lane >> 4;
  const int KB = a.K / 128;
  const int at = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3), item = part.first + at;
  if (at >= part.count) return;
  const int slab = item / part.tiles, t = item - slab * part.tiles;
  const Tile tile = find_tile<16 * kCT, 64 * kWaves>(a, t, part.tiles, lds.sh, &lds.tile);
  if (tile.rows <= 0) return;
  const int g = __builtin_amdgcn_readfirstlane(tile.g), m0 = __builtin_amdgcn_readfirstlane(tile.m0),
            rows = __builtin_amdgcn_readfirstlane(tile.rows), n0 = slab * 16 * kRT, nrows = min(16 * kRT, a.N - n0);
  const rsrc_t wr = make_rsrc(a.w + ((size_t)g * a.N + n0) * a.K, (size_t)nrows * a.K);
  const rsrc_t xr = make_rsrc(a.x + (size_t)m0 * a.x_stride, (size_t)(rows - 1) * a.x_stride + a.K);
  // LDS row 16 rt + m of the weights holds row 4 kRT (m / 4) + 4 rt + m % 4 of the slab, so that a lane's tiles are 4 kRT
  // consecutive columns of y; rows past the last one read zeros
  uint32_t wo[2 * kRT], xo[2 * kCT];
#pragma unroll
  for (int j = 0; j < 2 * kRT; ++j) {
    const int r = 8 * j + (lane >> 3), m = r & 15, n = 4 * kRT * (m >> 2) + 4 * (r >> 4) + (m & 3);
    wo[j] = (uint32_t)n * (uint32_t)a.K + 16u * (uint32_t)((lane & 7) ^ ((r >> 1) & 7));
  }
#pragma unroll
  for (int j = 0; j < 2 * kCT; ++j) {
    const int r = 8 * j + (lane >> 3);
    xo[j] = (uint32_t)min(r, rows - 1) * (uint32_t)a.x_stride + 16u * (uint32_t)((lane & 7) ^ ((r >> 1) & 7));
  }
  uint8_t* ring = lds.main + w * L::kRing;
  const int blocks = KB > w ? (KB - w + kWaves - 1) / kWaves : 0;
  // loads past the last block count but fetch nothing: a lane offset of 2^31 lies past any buffer's end
  const auto fetch = [&](int i, int slot, int part, int parts) {
    const uint32_t k = i < blocks ? (uint32_t)(w + kWaves * i) * 128u : 0u, past = i < blocks ? 0u : 0x80000000u;
    uint8_t* to = ring + slot * L::kBlock;
#pragma unroll
    for (int j = kLoads * part / parts; j < kLoads * (part + 1) / parts; ++j) {
      if (j < 2 * kRT) lds_load16(wr, wo[j] + past, k, to + 1024 * j);
      else lds_load16(xr, xo[j - 2 * kRT] + past, k, to + 1024 * j);
    }
  };
  const int ss = KB | 1;
  // the scales first: they are waited for by all, the blocks by their own wave
  {
    const float* sw = a.w_sf + ((size_t)g * ((a.N + 127) / 128) + n0 / 128) * KB;
    const float* sx = a.x_sf + (size_t)m0 * KB;
    for (int i = tid; i < KB; i += 64 * kWaves) lds.sw[i] = sw[i];
    for (int i = tid; i < rows * KB; i += 64 * kWaves) {
      const int r = i / KB;
      lds.sx[r * ss + i - r * KB] = sx[i];
    }
  }
#pragma unroll
  for (int s = 0; s < kStages; ++s) fetch(s, s, 0, 1);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  pipeline_barrier();

  const int sw7 = (lr >> 1) & 7;
  const int lo = lr * 128 + 16 * (lg ^ sw7), hi = lr * 128 + 16 * ((lg | 4) ^ sw7);
  v4f acc[kRT][kCT];
#pragma unroll
  for (int r = 0; r < kRT; ++r)
#pragma unroll
    for (int c = 0; c < kCT; ++c) acc[r][c] = v4f{0.f, 0.f, 0.f, 0.f};
  int srow[kCT];                                 // rows past the tile's last repeat that one
#pragma unroll
  for (int c = 0; c < kCT; ++c) srow[c] = min(16 * c + lr, rows - 1) * ss;
  for (int i = 0, slot = 0; i < blocks; ++i) {
    wait_vmcnt<(kStages - 1) * kLoads>();
    asm volatile("" ::: "memory");
    const uint8_t* S = ring + slot * L::kBlock;
    const int b = w + kWaves * i;
    v8i A[kRT], B[kCT];
    float s[kCT];
    const float cw = lds.sw[b];
#pragma unroll
    for (int c = 0; c < kCT; ++c) {
      B[c] = lds_operand(S + lo, S + hi, 2048 * (kRT + c));
      s[c] = lds.sx[srow[c] + b];
    }
#pragma unroll
    for (int r = 0; r < kRT; ++r) A[r] = lds_operand(S + lo, S + hi, 2048 * r);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read: the place may be filled again
    __builtin_amdgcn_sched_barrier(0);
    // the loads go out between the MFMAs, which run meanwhile: each waits for its turn in the address unit
    v4f p[kCT][kRT];
#pragma unroll
    for (int c = 0; c < kCT; ++c) {
#pragma unroll
      for (int r = 0; r < kRT; ++r) p[c][r] = mfma_block(A[r], B[c]);
      __builtin_amdgcn_sched_barrier(0);
      fetch(i + kStages, slot, c, kCT);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int c = 0; c < kCT; ++c) {
      const float sc = s[c] * cw;
#pragma unroll
      for (int r = 0; r < kRT; ++r) acc[r][c] += p[c][r] * sc;
    }
    slot = slot + 1 == kStages ? 0 : slot + 1;
  }
  wait_vmcnt<0>();                               // the rings' places are taken by the sums
  __syncthreads();
  v4f* sums = reinterpret_cast<v4f*>(lds.main);
#pragma unroll
  for (int r = 0; r < kRT; ++r)
#pragma unroll
    for (int c = 0; c < kCT; ++c) sums[((w * kCT + c) * kRT + r) * 64 + lane] = acc[r][c];
  __syncthreads();
  for (int i = tid; i < kRT * kCT * 64; i += 64 * kWaves) {
    const int r = i % kRT, c = i / kRT / 64, l = i / kRT % 64;
    v4f v = sums[(c * kRT + r) * 64 + l];
#pragma unroll
    for (int u = 1; u < kWaves; ++u) v += sums[((u * kCT + c) * kRT + r) * 64 + l];
    const int row = 16 * c + (l & 15), n = n0 + 4 * kRT * (l >> 4) + 4 * r;
    if (row < rows && n < a.N)
      *reinterpret_cast<uint2*>(a.y + (size_t)(m0 + row) * a.y_stride + n) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  }
}

// A workgroup for every slab of weight rows and every tile that the groups may be cut into.
template <int kVariant, class F>
hipError_t launch(const ProductArgs& a, hipStream_t s, int threads, F* kernel) {
  constexpr ProductTile t = kProductTiles[kVariant];
  const int64_t items = product_items(t, a.M, a.N, a.G, a.offset != nullptr);
  for (int64_t first = 0; first < items; first += kProductGroups) {
    const int count = (int)std::min(items - first, kProductGroups);
    const ProductPart part{(int)up_div(a.N, t.n), (int)product_tiles(t, a.M, a.G, a.offset != nullptr), (int)first, count};
    hipLaunchKernelGGL(kernel, dim3((unsigned)(count + 7) / 8 * 8), dim3(threads), 0, s, a, part);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

template <int kVariant, int kWaves, int kStages>
hipError_t launch_split(const ProductArgs& a, hipStream_t s) {
  constexpr ProductTile t = kProductTiles[kVariant];
  return launch<kVariant>(a, s, 64 * kWaves, k_product_split<t.n / 16, t.m / 16, kWaves, kStages, t.most_blocks>);
}

template <int kVariant, int kNG, int kWN, int kKS, int kStages>
hipError_t launch_large(const ProductArgs& a, hipStream_t s) {
  using L = LargeLds<kNG, kWN, kKS, kStages>;
  static_assert(L::kBN == kProductTiles[kVariant].n && L::kBM == kProductTiles[kVariant].m, "");
  return launch<kVariant>(a, s, 512, k_product_large<kNG, kWN, kKS, kStages>);
}

}  // namespace

hipError_t launch_product(const ProductArgs& a, hipStream_t s) {
  switch (product_variant(a.M, a.N, a.K, a.G)) {
    case 0: return launch_split<0, 8, 4>(a, s);
    case 1: return launch_split<1, 8, 2>(a, s);
    case 2: return launch_split<2, 4, 3>(a, s);
    case 3: return launch_split<3, 4, 2>(a, s);
    case 4: return launch_split<4, 4, 2>(a, s);
    case 5: return launch_large<5, 1, 2, 1, 4>(a, s);
    case 6: return launch_large<6, 2, 2, 2, 3>(a, s);
    case 7: return launch_large<7, 2, 2, 1, 4>(a, s);
    case 8: return launch_large<8, 2, 4, 1, 3>(a, s);
    case 9: return launch_large<9, 4, 4, 1, 3>(a, s);
    default: return launch_large<10, 8, 4, 1, 2>(a, s);
  }
}

}  // namespace mm
