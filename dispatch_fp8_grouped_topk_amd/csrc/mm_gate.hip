// Gate product: logits[t, e] = sum_h x[t, h] w[e, h] with BF16 MFMA, float32 sums.
//
// Weights are the MFMA's A operand (rows are experts) and tokens its B operand (columns), so a lane
// ends with four consecutive experts of one token.  Float32 weights are split into three BF16 terms of
// 8 significant bits each (w = hi + mid + lo exactly, by truncation) and multiplied by three MFMAs
// into the same sum.  A few logits are dot products of rows instead, with float32 multiply-adds (k_gate_rows).
#include "mm_front.h"
#include "mm_gate_policy.h"

namespace mm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f mfma_bf16(const v4i& a, const v4i& b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The upper halves of two words: two BF16 by truncation.
__device__ __forceinline__ int upper_halves(int lo, int hi) {
  return (int)__builtin_amdgcn_perm((uint32_t)hi, (uint32_t)lo, 0x07060302u);
}

// What is left of a float32 once its upper half is taken off, exactly.
__device__ __forceinline__ int lower_part(int v) {
  return __builtin_bit_cast(int, __builtin_bit_cast(float, v) - __builtin_bit_cast(float, v & (int)0xFFFF0000));
}

// 8 float32 weights a lane as three BF16 operands whose sum they are.
__device__ __forceinline__ void split3(const v4i (&w)[2], v4i (&parts)[3]) {
  v4i lo = w[0], hi = w[1];
#pragma unroll
  for (int term = 0; term < 3; ++term) {
    parts[term] = v4i{upper_halves(lo[0], lo[1]), upper_halves(lo[2], lo[3]), upper_halves(hi[0], hi[1]),
                      upper_halves(hi[2], hi[3])};
    if (term == 2) break;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = lower_part(lo[i]);
      hi[i] = lower_part(hi[i]);
    }
  }
}

// A 16-byte load of each lane from a buffer into consecutive LDS bytes from the wave-uniform `lds` on.
// Offsets at or past the buffer's size read zeros.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)(uint32_t)bytes, 0x00020000);
}
__device__ __forceinline__ void lds_load16(rsrc_t r, uint32_t voff, uint32_t soff, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, (int)soff, 0, 0);
}
template <int kN>
__device__ __forceinline__ void wait_vmcnt() {
  __builtin_amdgcn_s_waitcnt((kN & 0xF) | ((kN >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// One workgroup per tile of kE experts x kT tokens (each 8, which fills half an MFMA operand, or a
// multiple of 16).  Its kW waves share K: wave w takes the steps of 64 columns w, w + kW, ..., each for
// the whole tile, through a ring of its own in LDS (kSW steps of weights, kSX of tokens), so the loop has no
// barrier; the waves' sums meet in LDS at the end.  A step's weights are taken in kP parts: while one
// part is multiplied the next one is read into registers, and its place in the ring is filled again
// at once.
//
// T 8192, H 7168, E 256 (BF16 weights) takes 47.9 us: 628 TFLOP/s, of 21 us at the rate of a large matrix
// product and 24 us for its bytes at that of a large copy.  Bound by fetching: 2.75 MB a compute unit,
// at 36 bytes a clock with half the compute units busy (32 us) and 23 with all, where token rows come from HBM
// through the same in-order queue (39 us when they lie in the last-level cache).  The matrix cores are
// busy a quarter of the time, LDS has no bank conflicts.  Waves that only fetch tokens, three steps ahead,
// gained 3%, a wave that touches token lines ahead of the others lost 12%.
//
// Rows are fetched as whole 128-byte lines (8 rows x 128 bytes a load): operands loaded straight into
// registers touch 64 bytes of 16 rows, and the L2 delivers lines, half of each for nothing.
// In LDS a row's eight 16-byte chunks are permuted by (row / 2) % 8, so that the 16 rows of an
// operand read fall into different banks.
template <bool kWF32, int kE, int kT, int kW, int kSW, int kSX, int kP>
__global__ __launch_bounds__(64 * kW) void k_gate(GateArgs a, int etiles, int ttiles, int experts_first) {
  constexpr int kWB = kWF32 ? 4 : 2;                     // bytes a weight
  constexpr int kHalves = kWF32 ? 2 : 1;                 // 128-byte lines of a weight row in a step
  constexpr int kM = (kE + 15) / 16, kN = (kT + 15) / 16, kMP = kM / kP;   // MFMA operands of a tile, of a part
  constexpr int kRows = kE / 8 / kP;                     // loads of eight weight rows in a part
  constexpr int kLX = kT / 8, kLP = kRows * kHalves, kLW = kP * kLP;       // loads of a step, of a part
  // Loads issued since a part's own when it is waited for (a step's tokens go out with its part 0):
  // the rest of that step, the steps between, and what the present step has issued before this part.
  static_assert(kSX >= kSW && kM % kP == 0 && (kP == 1 || kP % 2 == 0), "");
  constexpr int kLater0 = kLW - kLP + (kSW - 1) * (kLX + kLW), kLater = kLater0 + kLX;
  static_assert(kLater < 64, "vmcnt holds 6 bits");
  // Eight experts fill an MFMA operand with both halves of a step: rows 0 .. 7 are its columns 0 .. 31, rows 8 .. 15 its
  // columns 32 .. 63, read (and split) once.  Tokens are multiplied half by half into sums of their own, of
  // which rows 0 .. 7 and rows 8 .. 15 count; or, eight of them, are folded the same way, one MFMA does
  // both halves and the diagonal quarters count.  The two parts are added at the end.
  constexpr bool kFoldE = kE == 8, kFoldT = kFoldE && kT == 8;
  constexpr int kSubsW = kFoldE ? 1 : 2, kSubsX = kFoldT ? 1 : 2;
  static_assert(!kFoldE || kT <= 16, "");
  constexpr int kXBytes = kLX * 1024, kWBytes = kLW * 1024;
  constexpr int kRing = kSX * kXBytes + kSW * kWBytes;   // a wave's LDS
  constexpr int kSums = kM * kN * 1024;                  // a wave's sums
  __shared__ __align__(1024) char lds[kW * (kRing > kSums ? kRing : kSums)];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, lg = lane >> 4;
  const int per = gridDim.x >> 3;
  // Each XCD walks neighbouring tiles: either all expert tiles of a few token tiles, or all token
  // tiles of a few expert tiles.
  const long tile = (long)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (tile >= (long)etiles * ttiles) return;
  const int e0 = (int)(experts_first ? tile % etiles : tile / ttiles) * kE;
  const long t0 = (experts_first ? tile / etiles : tile % ttiles) * kT;
  char* ring = lds + wave * kRing;

  // buffers of this tile's rows (at most 2^30 bytes): rows past the last one are out of range and read
  // zeros, or repeat the first ones; neither is stored
  const int erows = min(kE, a.E - e0), trows = (int)min((long)kT, a.T - t0);
  const uint32_t wstride = (uint32_t)a.H * kWB, xstride = (uint32_t)(a.x_stride * 2);
  const rsrc_t wr = make_rsrc(static_cast<const char*>(a.w) + (size_t)e0 * wstride, (size_t)erows * wstride);
  const rsrc_t xr = make_rsrc(a.x + (size_t)t0 * a.x_stride, (size_t)(trows - 1) * xstride + (size_t)a.H * 2);
  // lane l of a load: row l / 8 of its eight, chunk l % 8 of the line in LDS, which holds the line's
  // chunk (l % 8) ^ (row / 2 % 8); rows 8 .. 15 of an operand are the odd loads
  const int sub = lane >> 3;
  uint32_t wlane[2], xlane[2];
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const uint32_t chunk = 16u * (uint32_t)((lane & 7) ^ (4 * o + (sub >> 1)));
    wlane[o] = (uint32_t)sub * wstride + chunk;
    xlane[o] = (uint32_t)sub * xstride + chunk;
  }
  // operand reads: row col, chunk c of its line; a tile of eight rows is read twice over, or folded
  const auto chunk_at = [&](int c, int rows) {
    const int r = rows == 8 ? col & 7 : col;
    return r * 128 + ((c ^ (r >> 1)) * 16);
  };

  const int all = a.H / 64, steps = all > wave ? (all - wave + kW - 1) / kW : 0;
  // Out of range is what lies at or past the buffer's size less the scalar offset, so the scalar offset
  // itself stays inside: loads of a step past the last one, which count but fetch nothing, get a lane
  // offset of 2^31 and scalar offset 0, and loads of eight rows that are all past the tile's last
  // take the first eight.
  // The XCDs start at different columns and wrap round, so that they do not all ask for the same columns of
  // their rows at once (2 to 4% at T 1024 to 8192).
  const int turn = (int)(blockIdx.x & 7) * steps >> 3;
  const auto beyond = [&](int i) { return i < steps ? 0u : 0x80000000u; };
  const auto column = [&](int i) {
    const int j = i + turn;
    return i < steps ? (uint32_t)(wave + kW * (j < steps ? j : j - steps)) : 0u;
  };
  const auto rows_at = [&](int r, int rows, uint32_t stride) { return r < rows ? (uint32_t)r * stride : 0u; };
  const auto fetch_w = [&](int i, int slot, int p) {
    const uint32_t k = column(i) * (128 * kHalves), out = beyond(i);
    char* to = ring + kSX * kXBytes + slot * kWBytes + p * kLP * 1024;
#pragma unroll
    for (int m = 0; m < kRows; ++m)
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        lds_load16(wr, wlane[m & 1] + out, k + 128 * h + rows_at(8 * (kRows * p + m), erows, wstride),
                   to + (h * kRows + m) * 1024);
  };
  const auto fetch_x = [&](int i, int slot) {
    const uint32_t k = column(i) * 128, out = beyond(i);
    char* to = ring + slot * kXBytes;
#pragma unroll
    for (int n = 0; n < kLX; ++n) lds_load16(xr, xlane[n & 1] + out, k + rows_at(8 * n, trows, xstride), to + n * 1024);
  };

  v4i X[2][kSubsX][kN], W[2][kSubsW][kMP][kHalves];
  const auto read_x = [&](int slot, v4i (&to)[kSubsX][kN]) {
    const char* xs = ring + slot * kXBytes;
#pragma unroll
    for (int s = 0; s < kSubsX; ++s)
#pragma unroll
      for (int n = 0; n < kN; ++n) to[s][n] = *reinterpret_cast<const v4i*>(xs + n * 2048 + chunk_at(4 * (kFoldT ? col >> 3 : s) + lg, kT));
  };
  const auto read_w = [&](int slot, int p, v4i (&to)[kSubsW][kMP][kHalves]) {
    const char* ws = ring + kSX * kXBytes + slot * kWBytes + p * kLP * 1024;
#pragma unroll
    for (int s = 0; s < kSubsW; ++s)
#pragma unroll
      for (int m = 0; m < kMP; ++m) {
        const int half = kFoldE ? col >> 3 : s;
        if constexpr (kWF32) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            to[s][m][h] = *reinterpret_cast<const v4i*>(ws + (half * kRows + 2 * m) * 1024 + chunk_at(2 * lg + h, kE));
        } else {
          to[s][m][0] = *reinterpret_cast<const v4i*>(ws + m * 2048 + chunk_at(4 * half + lg, kE));
        }
      }
  };

  v4f acc[kM][kN], acc_half = {0.f, 0.f, 0.f, 0.f};   // acc_half: a folded tile's second half of the columns
#pragma unroll
  for (int m = 0; m < kM; ++m)
#pragma unroll
    for (int n = 0; n < kN; ++n) acc[m][n] = v4f{0.f, 0.f, 0.f, 0.f};

  if (steps > 0) {
#pragma unroll
    for (int j = -kSX; j < 0; ++j) {
      fetch_x(j + kSX, j + kSX);
      if (j + kSW >= 0)
#pragma unroll
        for (int p = 0; p < kP; ++p) fetch_w(j + kSW, j + kSW, p);
    }
    int sw = 0, sx = 0;                            // the ring's slots of step i
    wait_vmcnt<kLater0>();
    asm volatile("" ::: "memory");
    read_x(0, X[0]);
    read_w(0, 0, W[0]);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    fetch_x(kSX, 0);
    fetch_w(kSW, 0, 0);
    for (int i0 = 0; i0 < steps; i0 += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = i0 + u;
        if (u == 1 && i >= steps) break;
        const int sx1 = sx + 1 == kSX ? 0 : sx + 1, sw1 = sw + 1 == kSW ? 0 : sw + 1;
#pragma unroll
        for (int p = 0; p < kP; ++p) {
          const int b = (u * kP + p) & 1;          // registers of this part
          if (p + 1 < kP) {
            wait_vmcnt<kLater>();
            asm volatile("" ::: "memory");
            read_w(sw, p + 1, W[b ^ 1]);
          } else {
            wait_vmcnt<kLater0>();
            asm volatile("" ::: "memory");
            read_x(sx1, X[u ^ 1]);
            read_w(sw1, 0, W[b ^ 1]);
          }
          __builtin_amdgcn_sched_barrier(0);
          v4i parts[3];                            // float32 weights: the operand's terms
#pragma unroll
          for (int s = 0; s < kSubsX; ++s)
#pragma unroll
            for (int m = 0; m < kMP; ++m) {
              const v4i(&w)[kHalves] = W[b][kFoldE ? 0 : s][m];
              if constexpr (kWF32) {
                if (!kFoldE || s == 0) split3(w, parts);
              }
#pragma unroll
              for (int n = 0; n < kN; ++n) {
                v4f& c = kFoldE && s == 1 ? acc_half : acc[p * kMP + m][n];
                if constexpr (kWF32) {
#pragma unroll
                  for (int term = 0; term < 3; ++term) c = mfma_bf16(parts[term], X[u][s][n], c);
                } else {
                  c = mfma_bf16(w[0], X[u][s][n], c);
                }
              }
            }
          __builtin_amdgcn_sched_barrier(0);
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read: the place may be filled again
          if (p + 1 < kP) {
            fetch_w(i + kSW, sw, p + 1);
          } else {
            fetch_x(i + 1 + kSX, sx1);
            fetch_w(i + 1 + kSW, sw1, 0);
          }
        }
        sx = sx1;
        sw = sw1;
      }
    }
  }

  wait_vmcnt<0>();                                 // this wave's loads into LDS have landed
  __syncthreads();                                 // and every other's: the rings become the sums
  v4f* sums = reinterpret_cast<v4f*>(lds);
#pragma unroll
  for (int m = 0; m < kM; ++m)
#pragma unroll
    for (int n = 0; n < kN; ++n)
      sums[(wave * kM * kN + m * kN + n) * 64 + lane] = kFoldE && !kFoldT && lg >= 2 ? acc_half : acc[m][n];
  __syncthreads();
  for (int j = wave; j < kM * kN; j += kW) {
    v4f sum = sums[j * 64 + lane];
#pragma unroll
    for (int w = 1; w < kW; ++w) sum += sums[(w * kM * kN + j) * 64 + lane];
    if constexpr (kFoldE) {                        // the lane of row + 8 and, folded, column + 8
#pragma unroll
      for (int w = 0; w < kW; ++w) sum += sums[w * 64 + ((lane + (kFoldT ? 40 : 32)) & 63)];
    }
    const int e = e0 + 16 * (j / kN) + 4 * lg;
    const long t = t0 + 16 * (j % kN) + col;
    if (t >= a.T || (kE == 8 && lg >= 2) || (kT == 8 && col >= 8)) continue;
    float* out = a.logits + (size_t)t * a.E + e;
    if ((a.E & 3) == 0) {
      if (e < a.E) *reinterpret_cast<v4f*>(out) = sum;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < a.E) out[i] = sum[i];
    }
  }
}

template <bool kWF32, int kE, int kT, int kW, int kSW, int kSX, int kP>
hipError_t launch(const GateArgs& a, hipStream_t s) {
  const int etiles = (a.E + kE - 1) / kE, ttiles = (int)(((long)a.T + kT - 1) / kT);
  const long grid = ((long)etiles * ttiles + 7) / 8 * 8;
  // an XCD's L2 takes in one operand whole and an eighth of the other: the smaller one whole
  const int experts_first = (long)a.E * (kWF32 ? 4 : 2) <= (long)a.T * 2;
  hipLaunchKernelGGL((k_gate<kWF32, kE, kT, kW, kSW, kSX, kP>), dim3((unsigned)grid), dim3(64 * kW), 0, s, a, etiles, ttiles,
                     experts_first);
  return hipGetLastError();
}

// Products of few tokens: a workgroup for an expert and kT tokens, its lanes along their rows, straight
// from memory to registers, 8192 columns in flight at once, so that a row is one memory latency; the
// sums of 256 lanes are joined at the end.  Every term is one float32 multiply-add with the weight as it
// stands (float32 too), rounded once.  What bounds it is that latency and, with more tokens, the rows read
// again from L2.
template <bool kWF32, int kT>
__global__ __launch_bounds__(256) void k_gate_rows(GateArgs a) {
  constexpr int kB = 4, kWL = kWF32 ? 2 : 1;
  __shared__ float part[kT][4];
  const int tid = threadIdx.x, chunks = a.H / 8, e = blockIdx.x, t0 = blockIdx.y * kT;
  const v4i* wrow = reinterpret_cast<const v4i*>(static_cast<const char*>(a.w) + (size_t)e * a.H * (kWF32 ? 4 : 2));
  float acc[kT] = {};
  for (int c0 = 0; c0 < chunks; c0 += 256 * kB) {
    v4i w[kB][kWL], x[kB][kT];
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      const int c = c0 + 256 * b + tid;
#pragma unroll
      for (int l = 0; l < kWL; ++l) w[b][l] = v4i{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < kT; ++t) x[b][t] = v4i{0, 0, 0, 0};
      if (c < chunks) {
#pragma unroll
        for (int l = 0; l < kWL; ++l) w[b][l] = wrow[c * kWL + l];
#pragma unroll
        for (int t = 0; t < kT; ++t)
          x[b][t] = reinterpret_cast<const v4i*>(a.x + (size_t)min(t0 + t, a.T - 1) * a.x_stride)[c];
      }
    }
#pragma unroll
    for (int b = 0; b < kB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = w[b][0][i];                  // BF16 weights: a pair
        const int lo = kWF32 ? w[b][i / 2 * (kWL - 1)][2 * (i % 2)] : p << 16;
        const int hi = kWF32 ? w[b][i / 2 * (kWL - 1)][2 * (i % 2) + 1] : p & (int)0xFFFF0000;
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          const int u = x[b][t][i];
          acc[t] = __builtin_fmaf(__int_as_float(lo), __int_as_float(u << 16), acc[t]);
          acc[t] = __builtin_fmaf(__int_as_float(hi), __int_as_float(u & (int)0xFFFF0000), acc[t]);
        }
      }
  }
#pragma unroll
  for (int t = 0; t < kT; ++t) {
    const float sum = wave_sum63(acc[t]);
    if (tid % 64 == 63) part[t][tid / 64] = sum;
  }
  __syncthreads();
  if (tid < kT && t0 + tid < a.T)
    a.logits[(size_t)(t0 + tid) * a.E + e] = part[tid][0] + part[tid][1] + part[tid][2] + part[tid][3];
}

template <bool kWF32, int kT>
hipError_t launch_rows(const GateArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((k_gate_rows<kWF32, kT>), dim3(a.E, (a.T + kT - 1) / kT), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

// The choice of kernel and tile is gate_variant's (mm_gate_policy.h).
hipError_t launch_gate_logits(const GateArgs& a, hipStream_t s) {
  const int v = gate_variant(a.T, a.E, a.w_f32 != 0);
  if (v == kGateRowsSingle) return a.w_f32 ? launch_rows<true, 1>(a, s) : launch_rows<false, 1>(a, s);
  if (v == kGateRowsPair) return a.w_f32 ? launch_rows<true, 2>(a, s) : launch_rows<false, 2>(a, s);
  if (a.w_f32) {
    switch (v) {
      case 0: return launch<true, 8, 8, 8, 6, 6, 1>(a, s);
      case 1: return launch<true, 8, 16, 16, 2, 2, 1>(a, s);
      case 2: return launch<true, 16, 16, 8, 2, 2, 1>(a, s);
      case 3: return launch<true, 16, 32, 8, 2, 2, 1>(a, s);
      case 4: return launch<true, 32, 32, 8, 1, 1, 2>(a, s);
      case 5: return launch<true, 32, 64, 8, 1, 1, 2>(a, s);
      default: return launch<true, 64, 128, 4, 1, 1, 4>(a, s);
    }
  }
  switch (v) {
    case 0: return launch<false, 8, 8, 8, 9, 9, 1>(a, s);
    case 1: return launch<false, 8, 16, 8, 6, 6, 1>(a, s);
    case 2: return launch<false, 16, 16, 8, 4, 4, 1>(a, s);
    case 3: return launch<false, 16, 32, 8, 3, 3, 1>(a, s);
    case 4: return launch<false, 32, 32, 8, 2, 2, 1>(a, s);
    case 5: return launch<false, 64, 32, 8, 1, 2, 2>(a, s);
    case 6: return launch<false, 64, 64, 8, 1, 1, 2>(a, s);
    default: return launch<false, 128, 64, 4, 1, 2, 4>(a, s);
  }
}

}  // namespace mm
