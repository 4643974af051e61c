// Tokens sorted by expert and back: the plan (places of the pairs), the rows' way there, and the weighted way back with
// its gradient.  Everything moves rows of some kilobytes as 16-byte pieces, so the memory system is the bound; the plan
// is integers that depend on positions alone, never on the order in which atomics return.  A large copy reaches 5.1 TB/s
// here, reading alone 7.2, writing alone 6.9.
//
//   place of pair p with expert e:  #{pairs of experts below e} + #{pairs p' < p of e}
//   y[t] = sum_j w[t, j] rows[place(t, j)];  d_rows[place] = w dy[t];  d_w[t, j] = <rows[place], dy[t]>
#include "mm_parts.h"
#include "mm_route_dev.h"
#include "mm_rows.h"

namespace mm {
namespace {

// ------------------------------------------------------------------------------- small batches
// One launch: each workgroup moves one part of one token's row and finds the places of its k pairs itself, by
// counting the pairs that sort before each: with key(p) = expert * 4096 + p they are those with a smaller key.  A
// comparison of 64 pairs is one vector instruction and a count of bits, so 4096 pairs take 16 of them a wave and pair;
// that is cheaper than the other launches (E 256, k 8, 8-bit rows of 7168 columns: 511 tokens 13.0 us, 513 in blocks 14.9).
// The last workgroup makes expert_offset.  One token takes 4.4 us on the card: the launch, one memory latency for the ids and
// the row, two barriers, the stores.
template <bool kMove, int kIds>
__global__ __launch_bounds__(256) void k_sort_small(SortArgs a, int parts) {
  extern __shared__ int hist[];                  // [E], the last workgroup
  __shared__ int s_cnt[4][8], s_pos[8], sh[32];
  const int tid = threadIdx.x, wave = tid >> 6;
  // every id is asked for before anything that waits
  int ids[kIds];
#pragma unroll
  for (int i = 0; i < kIds; ++i) ids[i] = tid + 256 * i < a.P ? a.idx[tid + 256 * i] : -1;
  if ((int)blockIdx.x == a.T * parts) {
    for (int e = tid; e < a.E; e += 256) hist[e] = 0;
    __syncthreads();
    const auto count = [&](int e) {
      if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
    };
#pragma unroll
    for (int i = 0; i < kIds; ++i) count(ids[i]);
    __syncthreads();
    const int per = (a.E + 255) / 256, lo = min(tid * per, a.E), hi = min(lo + per, a.E);
    int sum = 0;
    for (int e = lo; e < hi; ++e) sum += hist[e];
    int v[1] = {sum}, all[1];
    block_scan_n<1, 256>(v, sh, all);
    int run = v[0] - sum;
    for (int e = lo; e < hi; ++e) {
      a.offset[e] = run;
      run += hist[e];
    }
    if (tid == 0) a.offset[a.E] = all[0];
    return;
  }
  const int t = blockIdx.x / parts, part = blockIdx.x - t * parts;
  // the first pieces of the row are asked for before the places are known
  const int chunks = a.row_bytes / 16, per = (chunks + parts - 1) / parts;
  const int c_lo = min(part * per, chunks), c_hi = min(c_lo + per, chunks);
  const uint4* from = reinterpret_cast<const uint4*>(static_cast<const char*>(a.x) + (size_t)t * a.x_stride);
  constexpr int kAhead = 4;
  uint4 v[kAhead];
  if constexpr (kMove) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int c = c_lo + tid + 256 * i;
      if (c < c_hi) v[i] = from[c];
    }
  }
  uint32_t word = 0;
  const bool scales = kMove && a.x_sf && part == 0 && tid < a.sf_words;
  if (scales) word = a.x_sf[(size_t)t * a.sf_words + tid];
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    uint32_t key[8], valid = 0;
    int cnt[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = j0 + j < a.k ? a.idx[t * a.k + j0 + j] : -1;
      const bool in = e >= 0 && e < a.E;
      key[j] = in ? (uint32_t)(e * kSortSmallPairs + t * a.k + j0 + j) : 0u;
      valid |= (uint32_t)in << j;
      cnt[j] = 0;
    }
    const auto compare = [&](int p, int e) {
      const uint32_t mine = e >= 0 && e < a.E ? (uint32_t)(e * kSortSmallPairs + p) : ~0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) cnt[j] += __popcll(__ballot(mine < key[j]));
    };
#pragma unroll
    for (int i = 0; i < kIds; ++i)
      if (256 * i < a.P) compare(tid + 256 * i, ids[i]);
    if ((tid & 63) == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s_cnt[wave][j] = cnt[j];
    }
    __syncthreads();
    if (tid < 8 && j0 + tid < a.k) {
      const int p = t * a.k + j0 + tid;
      const int at = (valid >> tid) & 1 ? s_cnt[0][tid] + s_cnt[1][tid] + s_cnt[2][tid] + s_cnt[3][tid] : -1;
      s_pos[tid] = at;
      if (part == 0) {
        a.pos[p] = at;
        if (at >= 0) a.src[at] = p;
      }
    }
    __syncthreads();
    if constexpr (kMove) {
      int at[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) at[j] = j0 + j < a.k ? __builtin_amdgcn_readfirstlane(s_pos[j]) : -1;
      const auto put = [&](int c, const uint4& piece) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at[j] >= 0)
            *reinterpret_cast<uint4*>(static_cast<char*>(a.rows) + (size_t)at[j] * a.row_bytes + 16 * (size_t)c) = piece;
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int c = c_lo + tid + 256 * i;
        if (c < c_hi) put(c, v[i]);
      }
      for (int c = c_lo + tid + 256 * kAhead; c < c_hi; c += 256) put(c, from[c]);
      if (scales) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at[j] >= 0) a.rows_sf[(size_t)at[j] * a.sf_words + tid] = word;
      }
    }
  }
}

// ------------------------------------------------------------------------------- large batches
// 1. Each block of block_pairs pairs: its pairs of each expert (blk), and each pair's rank among those of its expert in
// the block (in pos).  1024 pairs at a time: lanes of a wave with the same expert find each other bit by bit, and
// the waves add their counts to the histogram one after the other.
__global__ __launch_bounds__(1024) void k_sort_count(SortArgs a) {
  extern __shared__ int hist[];                  // [E]
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  for (int e = tid; e < a.E; e += 1024) hist[e] = 0;
  const int bits = 32 - __builtin_clz((unsigned)a.E);
  const int64_t lo = (int64_t)blockIdx.x * a.block_pairs, hi = min(lo + a.block_pairs, (int64_t)a.P);
  __syncthreads();
  for (int64_t base = lo; base < hi; base += 1024) {
    const int64_t p = base + tid;
    const int e = p < hi ? a.idx[p] : -1;
    const bool valid = e >= 0 && e < a.E;
    unsigned long long same = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
      const unsigned long long one = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? one : ~one;
    }
    const int before = __popcll(same & ((1ull << lane) - 1)), count = __popcll(same);
    int rank = -1;
    for (int w = 0; w < 16; ++w) {
      if (w == wave && valid) {
        const int h = hist[e];                   // every lane reads before the first of its expert adds
        rank = h + before;
        __builtin_amdgcn_wave_barrier();
        if (before == 0) hist[e] = h + count;
      }
      __syncthreads();
    }
    if (p < hi) a.pos[p] = rank;
  }
  for (int e = tid; e < a.E; e += 1024) a.blk[(size_t)blockIdx.x * a.E + e] = hist[e];
}

// 2. blk[b][e] becomes the pairs of e in blocks before b; total[e] those in all.  A workgroup takes 64 experts, its 16
// waves a sixteenth of the blocks each.
__global__ __launch_bounds__(1024) void k_sort_bases(SortArgs a) {
  __shared__ int part[16][64];
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6, e = blockIdx.x * 64 + lane;
  const int lo = (int)((int64_t)q * a.NB / 16), hi = (int)((int64_t)(q + 1) * a.NB / 16);
  int sum = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int b = lo; b < hi; ++b) sum += a.blk[(size_t)b * a.E + e];
  }
  part[q][lane] = sum;
  __syncthreads();
  if (e >= a.E) return;
  int run = 0;
  for (int i = 0; i < q; ++i) run += part[i][lane];
#pragma unroll 8
  for (int b = lo; b < hi; ++b) {
    const int c = a.blk[(size_t)b * a.E + e];
    a.blk[(size_t)b * a.E + e] = run;
    run += c;
  }
  if (q == 15) a.total[e] = run;
}

// 3. Places and rows: a wave takes a token, reads its row once and writes it k times, past the caches.  Every workgroup makes
// the experts' offsets from their totals itself (a kilobyte at 256 experts) rather than in a launch of their own.
// T 8192, H 7168, E 256, k 8 in BF16 (0.12 GB read, 0.91 written: 201 us at the rate of a large copy, 147 at those of reading
// and of writing alone) takes 208 us, and 9 for the two kernels before: bound by writing.  In all, stores through the caches
// took 328; the other way round, a wave a place that reads its token's row from the caches, 257 with stores past them and 310
// to 575 through them.
template <bool kMove>
__global__ __launch_bounds__(256) void k_sort_move(SortArgs a) {
  extern __shared__ int s_off[];                 // [E]
  __shared__ int sh[32];
  const int tid = threadIdx.x, lane = tid & 63;
  {
    const int per = (a.E + 255) / 256, lo = min(tid * per, a.E), hi = min(lo + per, a.E);
    int sum = 0;
    for (int e = lo; e < hi; ++e) sum += a.total[e];
    int v[1] = {sum}, all[1];
    block_scan_n<1, 256>(v, sh, all);
    int run = v[0] - sum;
    for (int e = lo; e < hi; ++e) {
      s_off[e] = run;
      if (blockIdx.x == 0) a.offset[e] = run;
      run += a.total[e];
    }
    if (blockIdx.x == 0 && tid == 0) a.offset[a.E] = all[0];
    __syncthreads();
  }
  const int chunks = a.row_bytes / 16;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (tid >> 6); t < a.T; t += (int64_t)gridDim.x * 4) {
    int at = -1;
    if (lane < a.k) {
      const int64_t p = t * a.k + lane;
      const int rank = a.pos[p];
      if (rank >= 0) {
        const int e = a.idx[p];
        at = s_off[e] + a.blk[(size_t)(p / a.block_pairs) * a.E + e] + rank;
        a.pos[p] = at;
        a.src[at] = (int)p;
      }
    }
    if constexpr (kMove) {
      const uint4* from = reinterpret_cast<const uint4*>(static_cast<const char*>(a.x) + (size_t)t * a.x_stride);
      if (__ballot(at >= 0) == 0) continue;
      constexpr int kPieces = 8;
      for (int c0 = 0; c0 < chunks; c0 += 64 * kPieces) {
        uint4 v[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          if (c0 + 64 * i + lane < chunks) v[i] = from[c0 + 64 * i + lane];
        for (int j = 0; j < a.k; ++j) {
          const int r = __builtin_amdgcn_readlane(at, j);
          if (r < 0) continue;
          uint4* to = reinterpret_cast<uint4*>(static_cast<char*>(a.rows) + (size_t)r * a.row_bytes);
#pragma unroll
          for (int i = 0; i < kPieces; ++i)
            if (c0 + 64 * i + lane < chunks) store16_nt(to + c0 + 64 * i + lane, v[i]);
        }
      }
      if (a.x_sf) {
        for (int c = lane; c < a.sf_words; c += 64) {
          const uint32_t word = a.x_sf[(size_t)t * a.sf_words + c];
          for (int j = 0; j < a.k; ++j) {
            const int r = __builtin_amdgcn_readlane(at, j);     // also of a lane without a word of its own
            if (r >= 0) a.rows_sf[(size_t)r * a.sf_words + c] = word;
          }
        }
      }
    }
  }
}

// kIds: ids a thread holds.  Fewer of them are less code to fetch, which is a part of what a single token takes.
template <int kIds>
void launch_small(const SortArgs& a, dim3 grid, int parts, size_t lds, hipStream_t s) {
  if (a.x) hipLaunchKernelGGL((k_sort_small<true, kIds>), grid, dim3(256), lds, s, a, parts);
  else hipLaunchKernelGGL((k_sort_small<false, kIds>), grid, dim3(256), lds, s, a, parts);
}

__global__ __launch_bounds__(256) void k_sort_empty(int32_t* offset, int n) {
  for (int e = blockIdx.x * 256 + threadIdx.x; e < n; e += gridDim.x * 256) offset[e] = 0;
}

}  // namespace

hipError_t launch_sort(const SortArgs& a, hipStream_t s) {
  if (a.T == 0) {
    hipLaunchKernelGGL(k_sort_empty, dim3((a.E + 256) / 256), dim3(256), 0, s, a.offset, a.E + 1);
    return hipGetLastError();
  }
  const size_t lds = (size_t)a.E * sizeof(int);
  if (a.P <= kSortSmallPairs) {
    // a token's row in up to four parts where there are fewer tokens than compute units
    int parts = 1;
    while (a.x && parts < 4 && (long)a.T * parts * 2 <= 512 && a.row_bytes / 16 > 256 * parts) parts *= 2;
    const dim3 grid((unsigned)(a.T * parts + 1));
    if (a.P <= 256) launch_small<1>(a, grid, parts, lds, s);
    else if (a.P <= 1024) launch_small<4>(a, grid, parts, lds, s);
    else launch_small<kSortSmallPairs / 256>(a, grid, parts, lds, s);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_sort_count, dim3((unsigned)a.NB), dim3(1024), lds, s, a);
  hipLaunchKernelGGL(k_sort_bases, dim3((unsigned)((a.E + 63) / 64)), dim3(1024), 0, s, a);
  const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)a.T + 3) / 4, 1 << 20);
  if (a.x) hipLaunchKernelGGL(k_sort_move<true>, dim3(grid), dim3(256), lds, s, a);
  else hipLaunchKernelGGL(k_sort_move<false>, dim3(grid), dim3(256), lds, s, a);
  return hipGetLastError();
}

namespace {

// ---------------------------------------------------------------------------------------- back
// A thread takes eight columns of a token: k places, then k pieces of rows under way at once, eight at a time, added up in
// ascending order.  T 4091, H 4096, k 8 in float32 (550 MB) takes 100 us, 5.5 TB/s (stores through the caches: 106), a decode
// batch of 128 x 7168 4.8 to 5.0 us on the card: two memory latencies after the launch.
template <bool kF32>
__global__ __launch_bounds__(256) void k_unsort(UnsortArgs a) {
  const int cpt = a.H / 8;
  const int64_t total = (int64_t)a.T * cpt;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / cpt;
    const int c = (int)(i - t * cpt);
    float acc[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) acc[n] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += 8) {
      int at[8];
      float w[8];
      Raw<kF32> v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = j0 + j < a.k;
        at[j] = in ? a.pos[t * a.k + j0 + j] : -1;
        w[j] = in && a.w ? a.w[t * a.k + j0 + j] : 1.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if ((uint32_t)at[j] < (uint32_t)a.R) v[j].load(a.rows, (size_t)at[j] * a.H + 8 * c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if ((uint32_t)at[j] >= (uint32_t)a.R) continue;
        float f[8];
        v[j].values(f);
#pragma unroll
        for (int n = 0; n < 8; ++n) acc[n] = __builtin_fmaf(w[j], f[n], acc[n]);
      }
    }
    store8_nt<kF32>(a.y, (size_t)t * a.stride + 8 * c, acc);
  }
}

// ---------------------------------------------------------------------------- back's gradient
// A workgroup takes a token, or for few tokens (kSplit) four of its pairs, its threads eight columns each (two times eight
// beyond 8192 columns): dy stays in registers,
// each pair's row is read once for d_w and written once.  Sums of eight products are float32, the rest of d_w's sum is
// float64: lanes by DPP, waves through LDS in a fixed order.  T 8192, H 7168, k 8 in BF16 (2.0 GB) takes 395 us, 5.1 TB/s;
// T 1021, H 4096 21.5 us, 6.0 TB/s (stores through the caches: 29.7).
constexpr int kAtOnce = 4;                       // pairs whose rows are under way at once
template <bool kF32, int kNC, bool kSplit>
__global__ __launch_bounds__(1024) void k_unsort_backward(UnsortArgs a) {
  __shared__ double part[16][kMaxTopk];
  const int chunks = a.H / 8, tid = threadIdx.x, waves = blockDim.x / 64;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    float d[kNC][8];
#pragma unroll
    for (int i = 0; i < kNC; ++i) {
      const int c = tid + i * blockDim.x;
      if (c >= chunks) continue;
      Raw<kF32> raw;
      raw.load(a.dy, (size_t)t * a.stride + 8 * c);
      raw.values(d[i]);
    }
    const int j_lo = kSplit ? blockIdx.y * kAtOnce : 0, j_hi = kSplit ? min(j_lo + kAtOnce, a.k) : a.k;
    for (int j0 = j_lo; j0 < j_hi; j0 += kAtOnce) {
      int at[kAtOnce];
      float w[kAtOnce];
      Raw<kF32> v[kAtOnce][kNC];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const bool in = j0 + j < a.k;
        at[j] = in ? a.pos[t * a.k + j0 + j] : -1;
        w[j] = in && a.w ? a.w[t * a.k + j0 + j] : 1.f;
        if ((uint32_t)at[j] >= (uint32_t)a.R) at[j] = -1;
      }
      if (a.d_w) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
          for (int i = 0; i < kNC; ++i) {
            const int c = tid + i * blockDim.x;
            if (at[j] >= 0 && c < chunks) v[j][i].load(a.rows, (size_t)at[j] * a.H + 8 * c);
          }
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (j0 + j >= a.k) continue;
        double dot = 0.0;
#pragma unroll
        for (int i = 0; i < kNC; ++i) {
          const int c = tid + i * blockDim.x;
          if (at[j] < 0 || c >= chunks) continue;
          if (a.d_w) {
            float f[8], sum = 0.f;
            v[j][i].values(f);
#pragma unroll
            for (int n = 0; n < 8; ++n) sum = __builtin_fmaf(f[n], d[i][n], sum);
            dot += (double)sum;
          }
          if (a.d_rows) {
            float o[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) o[n] = w[j] * d[i][n];
            store8_nt<kF32>(a.d_rows, (size_t)at[j] * a.H + 8 * c, o);
          }
        }
        if (a.d_w) {
          dot = wave_sum63(dot);
          if ((tid & 63) == 63) part[tid >> 6][j0 + j] = dot;
        }
      }
    }
    if (a.d_w) {
      __syncthreads();
      if (tid >= j_lo && tid < j_hi) {
        double dot = 0.0;
        for (int i = 0; i < waves; ++i) dot += part[i][tid];
        a.d_w[t * a.k + tid] = (float)dot;
      }
      __syncthreads();
    }
  }
}

// Below 512 tokens, two workgroups a compute unit, a token's pairs are shared out four by four (k 8, H 7168, us: T 1 7.1 -> 4.8,
// T 128 9.8 -> 7.5); above, that would only read dy again.
template <bool kF32, int kNC>
void launch_backward(const UnsortArgs& a, int threads, hipStream_t s) {
  if (a.T < 512)
    hipLaunchKernelGGL((k_unsort_backward<kF32, kNC, true>), dim3(a.T, (a.k + kAtOnce - 1) / kAtOnce), dim3(threads), 0, s, a);
  else
    hipLaunchKernelGGL((k_unsort_backward<kF32, kNC, false>), dim3(std::min(a.T, 1 << 20)), dim3(threads), 0, s, a);
}

template <bool kF32>
void launch_backward(const UnsortArgs& a, hipStream_t s) {
  const int chunks = a.H / 8, per = chunks <= 1024 ? 1 : 2, threads = ((chunks + per - 1) / per + 63) / 64 * 64;
  if (per == 1) launch_backward<kF32, 1>(a, threads, s);
  else launch_backward<kF32, 2>(a, threads, s);
}

}  // namespace

hipError_t launch_unsort(const UnsortArgs& a, hipStream_t s) {
  const int64_t total = (int64_t)a.T * (a.H / 8);
  const unsigned grid = (unsigned)std::min<int64_t>((total + 255) / 256, 1 << 20);
  if (a.f32) hipLaunchKernelGGL(k_unsort<true>, dim3(grid), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_unsort<false>, dim3(grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_unsort_backward(const UnsortArgs& a, hipStream_t s) {
  if (a.f32) launch_backward<true>(a, s);
  else launch_backward<false>(a, s);
  return hipGetLastError();
}

}  // namespace mm
