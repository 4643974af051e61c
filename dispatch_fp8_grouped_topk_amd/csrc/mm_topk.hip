// Choice of experts: scores, balance bias, expert groups, top-k and weights.
//
// One wave per row of logits.  Order is decided in float64, so that it does not depend on how an
// exponential is rounded: two scores that differ as real numbers compare as they do unless they lie
// within about 2^-50 of one another.  Without a bias the score is a monotone function of the logit and the
// logits themselves are compared.
//
// k_topk_wave holds the row in registers, up to 8 experts a lane, and k_topk_quarter four rows a wave, up to
// 16 experts a lane; k_topk_lds takes the rows that do not fit (more than 512 experts, or groups that
// leave too few lanes each) through LDS.
#include "mm_front.h"

namespace mm {
namespace {

constexpr double kNone = -__builtin_inf();       // ordering value of an expert that cannot be chosen

__device__ __forceinline__ float load_logit(const TopkArgs& a, size_t at) {
  if (a.bf16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[at] << 16);
  return static_cast<const float*>(a.logits)[at];
}

// NaN as -inf: not a candidate.
__device__ __forceinline__ float cleaned(float l) { return l == l ? l : -__builtin_inff(); }

struct Best {
  double v;
  int i;
};

// The larger value; of equal ones the lower index.
__device__ __forceinline__ Best better(Best a, Best b) {
  const bool take = b.v > a.v || (b.v == a.v && b.i < a.i);
  return take ? b : a;
}

__device__ __forceinline__ Best wave_best(Best b) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) b = better(b, Best{__shfl_xor(b.v, m), __shfl_xor(b.i, m)});
  return b;
}

// Scores of one row: sigmoid(l), or exp(l - top) / total.  l is not NaN.
struct Scorer {
  double top, inv_total;
  bool sigmoid;
  __device__ __forceinline__ double operator()(double l) const {
    if (sigmoid) return 1.0 / (1.0 + exp(-l));
    return (l == top ? 1.0 : exp(l - top)) * inv_total;
  }
};

__global__ __launch_bounds__(64) void k_topk_lds(TopkArgs a) {
  extern __shared__ double s_c[];                // [E] ordering values
  const int lane = threadIdx.x, cols = a.k + a.S, n = a.E / a.G;
  int valid = a.T;
  if (a.num_valid) valid = min(a.T, *a.num_valid);
  for (int row = blockIdx.x; row < a.T; row += gridDim.x) {
    int32_t* idx = a.idx + (size_t)row * cols;
    float* w = a.w + (size_t)row * cols;
    if (row >= valid) {
      for (int j = lane; j < cols; j += 64) {
        idx[j] = -1;
        w[j] = 0.f;
      }
      continue;
    }
    const size_t base = (size_t)row * a.stride;
    Scorer score{0.0, 0.0, a.sigmoid != 0};
    if (!a.sigmoid) {
      double top = kNone;
      for (int e = lane; e < a.E; e += 64) top = fmax(top, (double)cleaned(load_logit(a, base + e)));
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) top = fmax(top, __shfl_xor(top, m));
      double total = 0.0;
      for (int e = lane; e < a.E; e += 64) {
        const double l = cleaned(load_logit(a, base + e));
        if (l > kNone) total += l == top ? 1.0 : exp(l - top);
      }
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) total += __shfl_xor(total, m);
      score.top = top;
      score.inv_total = 1.0 / total;
    }
    __syncthreads();                             // the last row's values have been read
    for (int e = lane; e < a.E; e += 64) {
      const double l = cleaned(load_logit(a, base + e));
      double c = l;
      if (a.bias) {
        const float b = cleaned(a.bias[e]);
        c = l > kNone && b > -__builtin_inff() ? score(l) + (double)b : kNone;
      }
      s_c[e] = c;
    }
    __syncthreads();

    uint64_t kept = ~0ull;
    if (a.G > 1) {
      double v = kNone;
      if (lane < a.G) {
        double c1 = kNone, c2 = kNone;
        for (int i = 0; i < n; ++i) {
          const double c = s_c[lane * n + i];
          c2 = fmax(c2, fmin(c1, c));
          c1 = fmax(c1, c);
        }
        v = c1;
        if (a.group_top == 2 && c1 > kNone) {
          if (!a.bias) v = score(c1) + (c2 > kNone ? score(c2) : 0.0);
          else if (c2 > kNone) v = c1 + c2;
        }
      }
      kept = 0;
      for (int g = 0; g < a.KG; ++g) {
        const Best b = wave_best(Best{v, lane});
        if (!(b.v > kNone)) break;
        kept |= 1ull << b.i;
        if (lane == b.i) v = kNone;
      }
    }

    int mine = -1;                               // lane j: the j-th chosen expert
    for (int j = 0; j < a.k; ++j) {
      Best b{kNone, 1 << 30};
      for (int e = lane; e < a.E; e += 64) {
        if (a.G > 1 && !((kept >> (e / n)) & 1)) continue;
        b = better(b, Best{s_c[e], e});
      }
      b = wave_best(b);
      if (!(b.v > kNone)) break;
      if (lane == j) mine = b.i;
      if (lane == (b.i & 63)) s_c[b.i] = kNone;  // only this lane reads it again
    }
    double s = mine >= 0 ? score((double)load_logit(a, base + mine)) : 0.0;
    if (a.renorm) {
      double sum = s;
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
      s /= sum + 1e-20;
    }
    if (lane < a.k) {
      idx[lane] = mine;
      w[lane] = (float)(s * (double)a.scale);
    } else if (lane < cols) {
      idx[lane] = a.E + lane - a.k;
      w[lane] = a.shared_weight;
    }
  }
}

// exp(x) in float64 to about an ulp, for any x (NaN excepted): x = n ln 2 + r with |r| <= ln 2 / 2 (Cody and
// Waite's reduction), the Taylor series of exp(r) to r^13 / 13! (the next term is below 2^-57), times 2^n.
__device__ __forceinline__ double exp64(double x) {
  x = fmin(fmax(x, -800.0), 800.0);              // 2^n is 0 or infinity there
  const double n = __builtin_rint(x * 1.4426950408889634);
  // ln 2 in two parts, the first with 32 bits so that n times it is exact
  double r = __builtin_fma(n, -0.69314718036912382, x);
  r = __builtin_fma(n, -1.9082149292705877e-10, r);
  double p = 1.0 / 6227020800.0;
  p = __builtin_fma(p, r, 1.0 / 479001600.0);
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}

// Unsigned keys that order as the numbers do, 0 below every one of them (NaN and -inf are given 0).
__device__ __forceinline__ uint32_t key32(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 as +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value32(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t key64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
constexpr float kInf32 = __builtin_inff();

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)lane_value((uint32_t)(u >> 32), lane) << 32 | lane_value((uint32_t)u, lane));
}

// The value of a lane's partner in step `step` of a butterfly over 2, 4, 8, 16, 32 lanes.
__device__ __forceinline__ float dppf_xor(float v, int step) {
  const uint32_t u = __float_as_uint(v);
  switch (step) {
    case 0: return __uint_as_float(dpp<kXor1>(u));
    case 1: return __uint_as_float(dpp<kXor2>(u));
    case 2: return __uint_as_float(dpp<kHalfMirror>(u));
    case 3: return __uint_as_float(dpp<kMirror>(u));
    default: return __shfl_xor(v, 16);
  }
}
__device__ __forceinline__ double dppf_xor(double v, int step) {
  switch (step) {
    case 0: return dpp<kXor1>(v);
    case 1: return dpp<kXor2>(v);
    case 2: return dpp<kHalfMirror>(v);
    case 3: return dpp<kMirror>(v);
    default: return __shfl_xor(v, 16);
  }
}

// The two largest values of each group of 2^log2_lanes neighbouring lanes, from the lanes' two largest
// (-inf where there is none); at most half a wave.
template <class F>
__device__ __forceinline__ void best_two(F& m1, F& m2, int log2_lanes) {
#pragma unroll
  for (int step = 0; step < 5; ++step) {
    if (step >= log2_lanes) break;
    const F o1 = dppf_xor(m1, step), o2 = dppf_xor(m2, step);
    m2 = fmax(fmin(m1, o1), fmax(m2, o2));
    m1 = fmax(m1, o1);
  }
}

// A row's experts on the wave: kN a lane.  The lanes of a group are neighbours (2^log2_lanes of them), and
// experts go to lanes and places in ascending order, so that of equal values the lowest lane's lowest
// place is the lowest id.
struct Spread {
  int log2_lanes, n;                             // lanes and experts of a group
  __device__ __forceinline__ int first(int lane, int per) const {
    return (lane >> log2_lanes) * n + (lane & ((1 << log2_lanes) - 1)) * per;
  }
};

// Compare-exchange pairs of Batcher's odd-even merge sort of kN (a power of two) elements.
template <int kN>
struct Network {
  int lo[64] = {}, hi[64] = {}, count = 0;
  constexpr Network() {
    for (int p = 1; p < kN; p *= 2)
      for (int k = p; k >= 1; k /= 2)
        for (int j = k % p; j + k < kN; j += 2 * k)
          for (int i = 0; i < k && i + j + k < kN; ++i)
            if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
              lo[count] = i + j;
              hi[count] = i + j + k;
              ++count;
            }
  }
};

// Sorts pairs (key, low word) in descending order.
template <int kN, int kC = 0>
__device__ __forceinline__ void sort_pairs(uint32_t (&key)[kN], uint32_t (&low)[kN]) {
  constexpr Network<kN> net{};
  if constexpr (kC < net.count) {
    constexpr int x = net.lo[kC], y = net.hi[kC];
    const uint32_t kx = key[x], ky = key[y], lx = low[x], ly = low[y];
    const bool swap = ((uint64_t)ky << 32 | ly) > ((uint64_t)kx << 32 | lx);
    key[x] = swap ? ky : kx;
    key[y] = swap ? kx : ky;
    low[x] = swap ? ly : lx;
    low[y] = swap ? lx : ly;
    sort_pairs<kN, kC + 1>(key, low);
  }
}

// won ? next : here, as one bit select.  (Of two elements of an array the compiler makes one element at a
// chosen index, and of that a chain of compares.)
__device__ __forceinline__ uint32_t take_if(uint32_t won, uint32_t next, uint32_t here) { return (won & next) | (~won & here); }

// A lane's kN experts from `from` on, `mine` of them its own (the others are given -inf), NaN as -inf.
// whole: a lane has all of its kN or none, in one aligned piece.
template <int kN>
__device__ __forceinline__ void load_lane(const TopkArgs& a, size_t from, int mine, bool whole, float (&l)[kN]) {
  if (whole) {
    if (a.bf16) {
      uint16_t u[kN] = {};
      if (mine) __builtin_memcpy(u, __builtin_assume_aligned(static_cast<const uint16_t*>(a.logits) + from, kN * 2 < 16 ? kN * 2 : 16), kN * 2);
#pragma unroll
      for (int j = 0; j < kN; ++j) l[j] = __uint_as_float((uint32_t)u[j] << 16);
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) l[j] = 0.f;
      if (mine) __builtin_memcpy(l, __builtin_assume_aligned(static_cast<const float*>(a.logits) + from, kN * 4 < 16 ? kN * 4 : 16), kN * 4);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kN; ++j) l[j] = j < mine ? load_logit(a, from + j) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) l[j] = j < mine ? cleaned(l[j]) : -kInf32;
}
template <int kN>
__device__ __forceinline__ void load_bias(const TopkArgs& a, int e0, int mine, bool whole, float (&b)[kN]) {
#pragma unroll
  for (int j = 0; j < kN; ++j) b[j] = -kInf32;
  if (whole) {
    if (mine) __builtin_memcpy(b, __builtin_assume_aligned(a.bias + e0, kN * 4 < 16 ? kN * 4 : 16), kN * 4);
  } else {
#pragma unroll
    for (int j = 0; j < kN; ++j)
      if (j < mine) b[j] = a.bias[e0 + j];
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) b[j] = cleaned(b[j]);
}

// exp(x) to 2^-33, for weights, which are rounded to 2^-24; |x| at most 1000.  As exp64 with a shorter series, of which
// the terms from r^4 on, at most 2^-10 together, are float32, and as few steps after one another as it takes.
__device__ __forceinline__ double exp_weight(double x) {
  const double n = __builtin_rint(x * 1.4426950408889634), r = __builtin_fma(n, -0.6931471805599453, x), r2 = r * r;
  const float f = (float)r, f2 = f * f;
  const float a = __builtin_fmaf(f, 1.0f / 120.0f, 1.0f / 24.0f), b = __builtin_fmaf(f, 1.0f / 5040.0f, 1.0f / 720.0f),
              c = __builtin_fmaf(f, 1.0f / 362880.0f, 1.0f / 40320.0f);
  const float q = __builtin_fmaf(__builtin_fmaf(c, f2, b), f2, a);
  const double p = __builtin_fma(__builtin_fma((double)q, r2, __builtin_fma(r, 1.0 / 6.0, 0.5)), r2, 1.0 + r);
  return __builtin_ldexp(p, (int)n);
}

// 1 / y for a positive y whose reciprocal is a normal number: the hardware's estimate (2^-23) and a Newton step.
__device__ __forceinline__ double reciprocal64(double y) {
  const double e = __builtin_amdgcn_rcp(y);
  return __builtin_fma(__builtin_fma(-y, e, 1.0), e, e);
}

// The weight of a lane's chosen expert, 0 where it has none, in float64 so that it is rounded once, to float32.  top,
// total: the softmax's largest logit and its sum (0 where the scores decide nothing: it cancels under the renormalisation,
// and the chosen hold so much of it that 1e-20 does not count); sum_of: the sum over the row's lanes.  Exponents stop at
// +-700, beyond which a score is 0 or 1 all the same.
template <class Sum>
__device__ __forceinline__ double weight64(const TopkArgs& a, bool has, float logit, float top, double total, const Sum& sum_of) {
  double s = 0.0;
  if (has) {
    if (a.sigmoid) s = reciprocal64(1.0 + exp_weight(-(double)__builtin_amdgcn_fmed3f(logit, -700.f, 700.f)));
    else s = logit == top ? 1.0 : exp_weight(fmax((double)logit - (double)top, -700.0));     // infinities have no difference
  }
  if (a.renorm) total = sum_of(s) + (a.sigmoid ? 1e-20 : 1e-20 * total);
  else if (a.sigmoid) return s;
  return s > 0.0 ? s * reciprocal64(total) : 0.0;
}

// Whether two float32 ordering values may be out of order (see k_topk_wave).
struct Close {
  float step;                                    // at least twice the error of a score
  __device__ __forceinline__ bool operator()(float u, float v) const {
    return !(fabsf(u - v) > step + 0x1p-22f * fmaxf(fabsf(u), fabsf(v)));       // also where it is NaN
  }
  // How far a group's value, a sum of up to two biased scores, may be off, with as much again of what it rounds by:
  // two scores' errors, and 2^-23 of the biased scores' magnitudes, whose sum is `size`.
  __device__ __forceinline__ float of_group(float size) const { return step + 0x1p-22f * size; }
  static __device__ __forceinline__ Close of(bool sigmoid, float largest) { return {sigmoid ? 0x1p-20f : largest * 0x1p-16f}; }
};

// What a group's value lies between, as keys (0 where the group has no candidate).  The groups kept are the right
// ones if each one's lower end is above every dropped one's upper end.  Every group counts, not the two at the border
// alone: one whose two terms are large and cancel is off by their roundings wherever its sum stands in the order.
struct Ends {
  uint32_t lower, upper;
  __device__ __forceinline__ Ends(float v, float size, const Close& close) {
    const float off = close.of_group(size);      // an infinite size (an infinite bias, an overflow) leaves nothing sure
    lower = v == -kInf32 ? 0u : key32(off < kInf32 ? v - off : -kInf32);
    upper = v == -kInf32 ? 0u : key32(off < kInf32 ? v + off : kInf32);
  }
};

// One row's ordering values in float64: as keys (0: cannot be chosen), and the number of groups that come
// before this lane's.
template <int kN, class Score>
__device__ __forceinline__ int order64(const TopkArgs& a, const Spread& at, const float (&l)[kN], const float (&b)[kN],
                                       const Score& score, uint32_t (&hi)[kN], uint32_t (&lo)[kN]) {
  const int lane = threadIdx.x & 63, g = lane >> at.log2_lanes;
  double m1 = kNone, m2 = kNone;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    hi[j] = lo[j] = 0;
    if (l[j] > -kInf32 && b[j] > -kInf32) {
      const double c = a.bias ? score(l[j]) + (double)b[j] : (double)l[j];
      const uint64_t k = key64(c);
      hi[j] = (uint32_t)(k >> 32);
      lo[j] = (uint32_t)k;
      m2 = fmax(m2, fmin(m1, c));
      m1 = fmax(m1, c);
    }
  }
  if (a.G == 1) return 0;
  best_two(m1, m2, at.log2_lanes);
  double v = m1;
  if (a.group_top == 2 && m1 > kNone) {
    if (a.bias) v = m2 > kNone ? m1 + m2 : m1;
    else v = score((float)m1) + (m2 > kNone ? score((float)m2) : 0.0);
  }
  int rank = 0;
  for (int o = 0; o < a.G; ++o) {
    const double u = lane_value(v, o << at.log2_lanes);
    rank += u > v || (u == v && o < g);
  }
  return rank;
}

// The exact choice of one row, with values and comparisons in float64, for rows that float32 does not
// settle.  Returns the expert chosen r-th in lane r, -1 where there is none.
template <int kN, class Score>
__device__ __forceinline__ int choose64(const TopkArgs& a, const Spread& at, const float (&l)[kN], const float (&b)[kN],
                                        const Score& score) {
  const int lane = threadIdx.x & 63;
  uint32_t hi[kN], lo[kN];
  if (order64(a, at, l, b, score, hi, lo) >= a.KG) {
#pragma unroll
    for (int j = 0; j < kN; ++j) hi[j] = lo[j] = 0;
  }
  int chosen = -1;
  for (int r = 0; r < a.k; ++r) {
    uint64_t best = 0;
    int bj = 0;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const uint64_t k = (uint64_t)hi[j] << 32 | lo[j];
      bj = k > best ? j : bj;
      best = k > best ? k : best;
    }
    const uint32_t bh = (uint32_t)(best >> 32), bl = (uint32_t)best;
    const uint32_t mh = lane_value(wave_max63(bh), 63);
    if (mh == 0) break;                          // nothing left to choose
    const uint32_t ml = lane_value(wave_max63(bh == mh ? bl : 0u), 63);
    const int winner = __builtin_ctzll(__ballot(bh == mh && bl == ml));
    const int j = __builtin_amdgcn_readlane(bj, winner);
    if (lane == r) chosen = at.first(winner, kN) + j;
#pragma unroll
    for (int q = 0; q < kN; ++q)
      if (lane == winner && q == j) hi[q] = lo[q] = 0;
  }
  return chosen;
}

// A lane's part of the softmax's sum, in float32: each term is off by up to (1 + |l - lmax|) 2^-23 of itself (the
// difference and its product with log2 e are rounded, the exponential by a unit in the last place), their sum by
// log2(kN) roundings.  The mean of |l - lmax| over the whole softmax is at most its entropy, so with lanes joined in
// float64 the sum is off by less than (1 + ln 512 + 2) 2^-23 < 2^-19 of itself, and far less as errors vary: what does
// not is the rounding of log2 e, which therefore has a second part (worst weight of 4096 x 256 off by 1.0e-7 of itself
// instead of 1.2e-7, root mean square 2.9e-8 instead of 4.0e-8, of which the rounding to float32 is 2.5e-8).
template <int kN>
__device__ __forceinline__ float lane_sum(const float (&l)[kN], float lmax) {
  float t[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const float x = l[j] - lmax;
    t[j] = l[j] == lmax ? 1.f : __builtin_amdgcn_exp2f(__builtin_fmaf(x, 1.44269502f, x * 1.92596299e-8f));
  }
#pragma unroll
  for (int n = kN / 2; n > 0; n /= 2)
#pragma unroll
    for (int j = 0; j < n; ++j) t[j] += t[j + n];
  return t[0];
}

// One wave per row, kN experts a lane.  Each round takes the largest key of the wave: a DPP maximum and a
// ballot for the first lane that has it; lanes of up to four experts keep them sorted, and a round
// moves the winner's up.
//
// With a bias (kBiased), and for groups valued by two experts, scores are first computed in float32, whose
// error is bounded: a sigmoid's is below 2^-22 (the exponential's and the reciprocal's last places and
// three roundings), a softmax's below 2^-18 of the largest score (40 units in the last place for a sum
// of up to 1024 exponentials), the sum with the bias rounds by 2^-24 of itself.  Values further apart than
// at least twice these errors (Close) are in the right order.  So k + 2 experts are taken: where neighbours
// among the first k + 1 are close, those are ordered again by their float64 values, one a lane; where
// the k-th, k + 1-st and k + 2-nd are close to one another, the whole row is decided again in float64
// (choose64).  On random rows of 256 experts the former is one row in several hundred, the latter one in ten
// thousand.  Where a group that is dropped may be above one that is kept (Ends), the groups' order is decided
// in float64 (order64).  Without a bias the logits are compared, which is exact.
template <int kN, bool kBiased>
__global__ __launch_bounds__(256) void k_topk_wave(TopkArgs a, int log2_lanes, int vec) {
  const int lane = threadIdx.x & 63, cols = a.k + a.S;
  const Spread at{log2_lanes, a.E / a.G};
  const int g = lane >> log2_lanes, i0 = (lane & ((1 << log2_lanes) - 1)) * kN, e0 = at.first(lane, kN);
  const int mine = g < a.G ? min(max(at.n - i0, 0), kN) : 0;                // this lane's experts
  const bool by_score = kBiased || (a.G > 1 && a.group_top == 2);           // scores decide something
  for (int row = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); row < a.T; row += gridDim.x * 4) {
    int32_t* idx = a.idx + (size_t)row * cols;
    float* w = a.w + (size_t)row * cols;
    if (a.num_valid && row >= *a.num_valid) {
      if (lane < cols) {
        idx[lane] = -1;
        w[lane] = 0.f;
      }
      continue;
    }
    float l[kN], b[kN];
    load_lane(a, (size_t)row * a.stride + e0, mine, vec, l);
    if constexpr (kBiased) load_bias(a, e0, mine, vec, b);
    else
#pragma unroll
      for (int j = 0; j < kN; ++j) b[j] = 0.f;

    // the softmax's largest logit and, where scores are asked for, its sum
    float lmax = 0.f, unit = 1.f;                // unit: the largest score
    double sum32 = 0.0;
    if (!a.sigmoid) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < kN; ++j) top = max(top, l[j] > -kInf32 ? key32(l[j]) : 0u);
      const uint32_t k = lane_value(wave_max63(top), 63);
      lmax = k ? value32(k) : 0.f;
      if (by_score || !a.renorm) {
        sum32 = lane_value(wave_sum63((double)lane_sum(l, lmax)), 63);
        unit = __builtin_amdgcn_rcpf((float)sum32);
      }
    }
    const auto score32 = [&](float v) -> float {
      if (a.sigmoid) return __builtin_amdgcn_rcpf(1.f + __expf(-v));
      return (v == lmax ? 1.f : __expf(v - lmax)) * unit;
    };

    uint32_t key[kN];
    float m1 = -kInf32, m2 = -kInf32;            // the lane's two largest ordering values
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      float c = l[j];
      if constexpr (kBiased) c = l[j] > -kInf32 && b[j] > -kInf32 ? score32(l[j]) + b[j] : -kInf32;
      key[j] = c > -kInf32 ? key32(c) : 0u;
      m2 = fmaxf(m2, fminf(m1, c));
      m1 = fmaxf(m1, c);
    }

    // the same in float64, for the rare rows that need it
    const auto part64 = [&](float v) -> double { return v == lmax ? 1.0 : exp64((double)v - (double)lmax); };
    double total = 0.0;
    const auto need_total = [&] {
      if (a.sigmoid || total > 0.0) return;
      double t = 0.0;
#pragma unroll
      for (int j = 0; j < kN; ++j) t += part64(l[j]);
      total = lane_value(wave_sum63(t), 63);
    };
    const auto score64 = [&](float v) -> double {
      if (a.sigmoid) return 1.0 / (1.0 + exp64(-(double)v));
      return part64(v) / total;
    };
    const Close close = Close::of(a.sigmoid, unit);
    if (a.G > 1) {
      best_two(m1, m2, log2_lanes);
      float v = m1, size = fabsf(m1);            // size: the magnitudes of what v is the sum of
      if (a.group_top == 2 && m1 > -kInf32) {
        if constexpr (kBiased) {
          v = m2 > -kInf32 ? m1 + m2 : m1;
          size = m2 > -kInf32 ? fabsf(m1) + fabsf(m2) : fabsf(m1);
        } else {
          size = v = score32(m1) + (m2 > -kInf32 ? score32(m2) : 0.f);
        }
      }
      int rank = 0;                              // groups that come before this lane's
      for (int o = 0; o < a.G; ++o) {
        const float u = __uint_as_float(lane_value(__float_as_uint(v), o << log2_lanes));
        rank += u > v || (u == v && o < g);
      }
      if (by_score) {
        // the least of the kept groups' lower ends, the largest of the dropped groups' upper ends
        const Ends ends(v, size, close);
        const uint32_t out = lane_value(wave_max63(rank >= a.KG && g < a.G ? ends.upper : 0u), 63);
        if (out && ~lane_value(wave_max63(rank < a.KG && g < a.G ? ~ends.lower : 0u), 63) <= out) {
          uint32_t hi[kN], lo[kN];
          need_total();
          rank = order64(a, at, l, b, score64, hi, lo);
        }
      }
      if (rank >= a.KG) {
#pragma unroll
        for (int j = 0; j < kN; ++j) key[j] = 0;
      }
    }

    constexpr bool kSorted = kN <= 4;
    uint32_t place[kN];                          // of equal keys the lower place, which is the larger here, first
#pragma unroll
    for (int j = 0; j < kN; ++j) place[j] = kN - 1 - j;
    if constexpr (kSorted) sort_pairs(key, place);
    int chosen = -1, source = 0;                 // lane r: the expert chosen r-th, its lane and place
    uint32_t taken = 0;                          // and its key; two more where closeness matters
    const int rounds = kBiased ? a.k + 2 : a.k;
    for (int r = 0; r < rounds; ++r) {
      uint32_t best = key[0];
      int bj = kSorted ? kN - 1 - (int)place[0] : 0;
      if constexpr (!kSorted) {
#pragma unroll
        for (int j = 1; j < kN; ++j) {
          bj = key[j] > best ? j : bj;
          best = max(best, key[j]);
        }
      }
      const uint32_t m = lane_value(wave_max63(best), 63);
      if (m == 0) break;                         // nothing left to choose
      const int winner = __builtin_ctzll(__ballot(best == m));
      const int j = __builtin_amdgcn_readlane(bj, winner);
      if (lane == r) {
        chosen = at.first(winner, kN) + j;
        source = winner << 8 | j;
        taken = m;
      }
      if constexpr (kSorted) {
        const uint32_t won = lane == winner ? ~0u : 0u;
#pragma unroll
        for (int q = 0; q + 1 < kN; ++q) {
          key[q] = take_if(won, key[q + 1], key[q]);
          place[q] = take_if(won, place[q + 1], place[q]);
        }
        key[kN - 1] &= ~won;
      } else {
#pragma unroll
        for (int q = 0; q < kN; ++q) key[q] = lane == winner && q == j ? 0u : key[q];
      }
    }
    float logit = 0.f;
    const auto fetch_logit = [&] {
      if (!kBiased) {                            // the key says it
        logit = value32(taken);
        return;
      }
#pragma unroll
      for (int p = 0; p < kN; ++p) {
        const float v = __shfl(l[p], source >> 8);
        logit = p == (source & 0xFF) ? v : logit;
      }
    };
    fetch_logit();

    if constexpr (kBiased) {
      const uint32_t next = __shfl_down(taken, 1);
      const bool near = lane <= a.k && lane < 63 && taken && next && close(value32(taken), value32(next));
      const bool redo = a.k > 62;                // k + 2 do not fit the lanes
      const uint64_t nears = __ballot(near);
      if (redo || (nears & ((1ull << a.k) - 1))) {
        need_total();
        if (redo || ((nears >> (a.k - 1)) & 3) == 3) {
          chosen = choose64<kN>(a, at, l, b, score64);
          const int q = chosen < 0 ? 0 : chosen, qg = q / at.n, qi = q - qg * at.n;
          source = ((qg << log2_lanes) + qi / kN) << 8 | qi % kN;
        } else {
          const bool has = lane <= a.k && chosen >= 0;
          double c = kNone;
          if (has) c = score64(logit) + (double)a.bias[chosen];
          int rank = 0;
          for (int o = 0; o <= a.k; ++o) {
            const double u = lane_value(c, o);
            const int e = __builtin_amdgcn_readlane(chosen, o);
            rank += u > c || (u == c && e < chosen);
          }
          const int to = (has ? rank : lane) * 4;  // a lane without an expert stays behind those with one
          chosen = __builtin_amdgcn_ds_permute(to, chosen);
          source = __builtin_amdgcn_ds_permute(to, source);
        }
        fetch_logit();
      }
    }
    if (lane >= a.k) chosen = -1;

    const double s = weight64(a, chosen >= 0, logit, lmax, sum32, [](double v) { return lane_value(wave_sum63(v), 63); });
    if (lane < a.k) {
      idx[lane] = chosen;
      w[lane] = (float)(s * (double)a.scale);
    } else if (lane < cols) {
      idx[lane] = a.E + lane - a.k;
      w[lane] = a.shared_weight;
    }
  }
}

// Largest / sum over the 16 lanes of a DPP row, in all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  return max(v, dpp<kMirror>(v));
}
template <class F>
__device__ __forceinline__ F row_sum(F v) {
#pragma unroll
  for (int step = 0; step < 4; ++step) v += dppf_xor(v, step);
  return v;
}
template <int kN>
struct Rotations {                               // f(n) for n = kN - 1 .. 1 as compile-time constants
  template <class Fn>
  static __device__ __forceinline__ void each(Fn&& f) {
    f(Ctrl<kN - 1>{});
    if constexpr (kN > 2) Rotations<kN - 1>::each(f);
  }
};

// As k_topk_wave for many rows: four rows a wave, one on each 16 lanes, kN experts a lane, so that what
// a row costs besides its experts is shared by four.  Each lane's keys are sorted once; a round takes the
// row's largest head by a DPP maximum, and the lane that has it moves its keys up and leaves the expert
// in LDS.  T 8192, E 256, k 8 of 4 of 8 groups, sigmoid and bias: 10.7 us, of which an empty launch is 2; bound
// by the length of one wave's chain (1600 vector and 480 scalar instructions for its four rows) at two waves a SIMD.
template <int kN, bool kBiased>
__global__ __launch_bounds__(256) void k_topk_quarter(TopkArgs a, int log2_lanes, int vec) {
  __shared__ int s_chosen[4][4][16];             // by wave and row: the experts chosen; the groups kept
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, quarter = lane >> 4, li = lane & 15, cols = a.k + a.S;
  const Spread at{log2_lanes, a.E / a.G};
  const int g = li >> log2_lanes, i0 = (li & ((1 << log2_lanes) - 1)) * kN, e0 = at.first(li, kN);
  const int lane_experts = g < a.G ? min(max(at.n - i0, 0), kN) : 0;
  const bool by_score = kBiased || (a.G > 1 && a.group_top == 2);
  const int valid = a.num_valid ? min(a.T, *a.num_valid) : a.T;
  int* out = s_chosen[wave][quarter];
  for (int row0 = (blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(wave)) * 4; row0 < a.T; row0 += gridDim.x * 16) {
    const int row = row0 + quarter;
    const int mine = row < valid ? lane_experts : 0;         // padding is not looked at
    const size_t base = (size_t)min(row, a.T - 1) * a.stride;
    float l[kN];
    load_lane(a, base + e0, mine, vec, l);
    float b[kN];
    if constexpr (kBiased) load_bias(a, e0, mine, vec, b);

    float lmax = 0.f, unit = 1.f;
    double sum32 = 0.0;
    if (!a.sigmoid) {
      float top = l[0];
#pragma unroll
      for (int j = 1; j < kN; ++j) top = fmaxf(top, l[j]);
      const uint32_t k = row_max(top > -kInf32 ? key32(top) : 0u);
      lmax = k ? value32(k) : 0.f;
      if (by_score || !a.renorm) {
        sum32 = row_sum((double)lane_sum(l, lmax));
        unit = __builtin_amdgcn_rcpf((float)sum32);
      }
    }
    const auto part64 = [&](float v) -> double { return v == lmax ? 1.0 : exp64((double)v - (double)lmax); };
    const auto score32 = [&](float v) -> float {
      if (a.sigmoid) return __builtin_amdgcn_rcpf(1.f + __expf(-v));
      return (v == lmax ? 1.f : __expf(v - lmax)) * unit;
    };

    uint32_t key[kN];
    float m1 = -kInf32, m2 = -kInf32;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      float c = l[j];
      if constexpr (kBiased) {
        c = l[j] > -kInf32 && b[j] > -kInf32 ? score32(l[j]) + b[j] : -kInf32;
      }
      key[j] = c > -kInf32 ? key32(c) : 0u;
      m2 = fmaxf(m2, fminf(m1, c));
      m1 = fmaxf(m1, c);
    }

    // f(spread, l, b, score) for row q of the wave's four with the row on all 64 lanes, four experts each, and
    // scores in float64: for the rare rows that need it
    const auto on_wave = [&](int q, auto&& f) {
      int log2_wide = 6;
      while ((a.G << log2_wide) > 64) --log2_wide;
      const Spread wide{log2_wide, at.n};
      const int w0 = (lane & ((1 << log2_wide) - 1)) * 4, we = wide.first(lane, 4);
      const int has = (lane >> log2_wide) < a.G ? min(max(at.n - w0, 0), 4) : 0;
      float l4[4], b4[4] = {};
      load_lane(a, (size_t)(row0 + q) * a.stride + we, has, false, l4);
      if constexpr (kBiased) load_bias(a, we, has, false, b4);
      double lm = 0.0, total = 1.0;
      if (!a.sigmoid) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, l4[j] > -kInf32 ? key32(l4[j]) : 0u);
        const uint32_t k = lane_value(wave_max63(top), 63);
        lm = k ? (double)value32(k) : 0.0;
        double t = 0.0;
#pragma unroll
        for (int j = 0; j < 4; ++j) t += (double)l4[j] == lm ? 1.0 : exp64((double)l4[j] - lm);
        total = lane_value(wave_sum63(t), 63);
      }
      f(wide, l4, b4, [&](float v) -> double {
        if (a.sigmoid) return 1.0 / (1.0 + exp64(-(double)v));
        return ((double)v == lm ? 1.0 : exp64((double)v - lm)) / total;
      });
    };
    const auto lds_done = [] {                   // this wave's writes to LDS are there for its other lanes
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    };
    const Close close = Close::of(a.sigmoid, unit);
    if (a.G > 1) {
      best_two(m1, m2, log2_lanes);
      float v = m1, size = fabsf(m1);            // size: the magnitudes of what v is the sum of
      if (a.group_top == 2 && m1 > -kInf32) {
        if constexpr (kBiased) {
          v = m2 > -kInf32 ? m1 + m2 : m1;
          size = m2 > -kInf32 ? fabsf(m1) + fabsf(m2) : fabsf(m1);
        } else {
          size = v = score32(m1) + (m2 > -kInf32 ? score32(m2) : 0.f);
        }
      }
      if (g >= a.G) v = -kInf32;
      int before = 0;                            // lanes of the groups that come before this lane's
      Rotations<16>::each([&](auto n) {
        const float u = __uint_as_float(dpp<kRor + decltype(n)::value>(__float_as_uint(v)));   // of lane li - n
        const int og = ((li - decltype(n)::value) & 15) >> log2_lanes;
        before += u > v || (u == v && og < g);
      });
      bool kept = before < a.KG << log2_lanes;
      if (by_score) {
        // the least of the kept groups' lower ends, the largest of the dropped groups' upper ends
        const Ends ends(v, size, close);
        const uint32_t last = ~row_max(kept ? ~ends.lower : 0u), first = row_max(kept ? 0u : ends.upper);
        const uint64_t which = __ballot(row < valid && first != 0 && last <= first);
        if (which) {
          for (int q = 0; q < 4; ++q) {
            if (!((which >> (16 * q)) & 0xFFFF)) continue;
            on_wave(q, [&](const Spread& wide, const float(&l4)[4], const float(&b4)[4], const auto& score) {
              uint32_t hi[4], lo[4];
              const int rank = order64(a, wide, l4, b4, score, hi, lo), wg = lane >> wide.log2_lanes;
              if (wg < a.G) s_chosen[wave][q][wg] = rank < a.KG;
            });
          }
          lds_done();
          if (((which >> (16 * quarter)) & 0xFFFF) && g < a.G) kept = out[g] != 0;
          lds_done();
        }
      }
      if (!kept) {
#pragma unroll
        for (int j = 0; j < kN; ++j) key[j] = 0;
      }
    }

    // sort the keys with their places; of equal keys the lower place first
    uint64_t places = 0;                           // four bits a place, the next one lowest
    {
      uint32_t place[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) place[j] = kN - 1 - j;
      sort_pairs(key, place);
#pragma unroll
      for (int j = 0; j < kN; ++j) places |= (uint64_t)place[j] << (4 * j);
    }

    uint32_t taken = 0;                          // lane r: the key taken r-th, 0 where there was none
    const uint32_t below = (1u << li) - 1;
    const int rounds = kBiased ? a.k + 2 : a.k;
    for (int r = 0; r < rounds; ++r) {
      const uint32_t m = row_max(key[0]);
      const uint64_t who = __ballot(key[0] == m && m != 0);
      if (who == 0) break;
      const bool won = key[0] == m && m != 0 && ((uint32_t)(who >> (16 * quarter)) & below) == 0;
      if (li == r) taken = m;
      if (won) out[r] = e0 + kN - 1 - (int)(places & 15);
      const uint32_t mask = won ? ~0u : 0u;
#pragma unroll
      for (int q = 0; q + 1 < kN; ++q) key[q] = take_if(mask, key[q + 1], key[q]);
      key[kN - 1] &= ~mask;
      places >>= mask & 4;
    }
    lds_done();
    int chosen = taken ? out[li] : -1;
    float logit = value32(taken);                // without a bias the key says it
    if constexpr (kBiased) {
      logit = chosen >= 0 ? load_logit(a, base + chosen) : 0.f;
      const uint32_t next = dpp<kShl + 1>(taken);
      const bool near = li <= a.k && taken && next && close(value32(taken), value32(next));
      const uint32_t nears = (uint32_t)(__ballot(near && row < valid) >> (16 * quarter)) & 0xFFFF;
      const bool redo = ((nears >> (a.k - 1)) & 3) == 3, again = !redo && (nears & ((1u << a.k) - 1));
      if (__ballot(again)) {
        double total = 1.0;
        if (!a.sigmoid) {
          double t = 0.0;
#pragma unroll
          for (int j = 0; j < kN; ++j) t += part64(l[j]);
          total = row_sum(t);
        }
        const bool has = li <= a.k && chosen >= 0;
        double c = kNone;
        if (has) {
          const double b = a.bias[chosen];
          if (a.sigmoid) c = 1.0 / (1.0 + exp64(-(double)logit)) + b;
          else c = part64(logit) / total + b;
        }
        int rank = 0;
        Rotations<16>::each([&](auto n) {
          const double u = dpp<kRor + decltype(n)::value>(c);
          const int e = (int)dpp<kRor + decltype(n)::value>((uint32_t)chosen);
          rank += u > c || (u == c && e < chosen && u > kNone);
        });
        const int to = (again && has ? 16 * quarter + rank : lane) * 4;
        chosen = __builtin_amdgcn_ds_permute(to, chosen);
        logit = __builtin_bit_cast(float, __builtin_amdgcn_ds_permute(to, __builtin_bit_cast(int, logit)));
      }
      const uint64_t which = __ballot(redo);
      if (which) {
        lds_done();
        for (int q = 0; q < 4; ++q) {
          if (!((which >> (16 * q)) & 0xFFFF)) continue;
          on_wave(q, [&](const Spread& wide, const float(&l4)[4], const float(&b4)[4], const auto& score) {
            const int c = choose64<4>(a, wide, l4, b4, score);
            if (lane < a.k) s_chosen[wave][q][lane] = c;
          });
        }
        lds_done();
        if (redo && li < a.k) {
          chosen = out[li];
          logit = chosen >= 0 ? load_logit(a, base + chosen) : 0.f;
        }
      }
    }
    lds_done();                                  // read before the next rows' are written
    if (li >= a.k) chosen = -1;

    const double s = weight64(a, chosen >= 0, logit, lmax, sum32, [](double v) { return row_sum(v); });
    if (row < a.T && li < cols) {
      int e = chosen;
      float w = (float)(s * (double)a.scale);
      if (li >= a.k) e = a.E + li - a.k, w = a.shared_weight;
      if (row >= valid) e = -1, w = 0.f;
      a.idx[(size_t)row * cols + li] = e;
      a.w[(size_t)row * cols + li] = w;
    }
  }
}

template <int kN>
void launch_quarter(const TopkArgs& a, int log2_lanes, int vec, hipStream_t s) {
  const int groups = (a.T + 15) / 16, grid = groups < (1 << 20) ? groups : (1 << 20);
  if (a.bias) hipLaunchKernelGGL((k_topk_quarter<kN, true>), dim3(grid), dim3(256), 0, s, a, log2_lanes, vec);
  else hipLaunchKernelGGL((k_topk_quarter<kN, false>), dim3(grid), dim3(256), 0, s, a, log2_lanes, vec);
}

template <int kN>
void launch_wave(const TopkArgs& a, int log2_lanes, int vec, hipStream_t s) {
  const int groups = (a.T + 3) / 4, grid = groups < (1 << 20) ? groups : (1 << 20);
  if (a.bias) hipLaunchKernelGGL((k_topk_wave<kN, true>), dim3(grid), dim3(256), 0, s, a, log2_lanes, vec);
  else hipLaunchKernelGGL((k_topk_wave<kN, false>), dim3(grid), dim3(256), 0, s, a, log2_lanes, vec);
}

}  // namespace

hipError_t launch_gate_topk(const TopkArgs& a, hipStream_t s) {
  // each group has the same power of two of lanes, each lane `need` of its experts
  int log2_lanes = 6;
  while ((a.G << log2_lanes) > 64) --log2_lanes;
  const int n = a.E / a.G, need = (n + (1 << log2_lanes) - 1) >> log2_lanes;
  // a lane's experts are one aligned piece where its group's are whole lanes
  const auto vec = [&](int per) {
    const int bytes = per * (a.bf16 ? 2 : 4), piece = bytes < 16 ? bytes : 16;
    return n % per == 0 && a.stride * (a.bf16 ? 2 : 4) % piece == 0 ? 1 : 0;
  };
  int quarter_lanes = 4;
  while ((a.G << quarter_lanes) > 16 && quarter_lanes > 0) --quarter_lanes;
  const int quarter_need = (n + (1 << quarter_lanes) - 1) >> quarter_lanes;
  // Four rows a wave take longer for one row and less for many.  Measured (us, k 8, quarter against wave; sigmoid and
  // bias unless stated) at T 2048, 3000, 4096, 5000, 6000, 7000, 8192:
  //   E 64                      4.8 4.4, 4.9 4.8, 4.9 5.6, 5.2 6.0, 5.2 6.6, 5.2 7.4, 5.3 8.1
  //   E 64, softmax, no bias    3.6 3.7, 3.6 4.0, 3.6 4.5, 4.0 5.0, 4.0 5.4, 4.0 6.0, 4.1 6.5
  //   E 128                     5.5 4.8, 5.5 5.1, 5.5 6.1, 5.8 6.4, 6.3 7.2, 6.3 8.0, 6.3 8.8
  //   E 256                     8.1 5.5, 8.2 6.1, 8.2 7.0, 8.8 7.5, 9.0 8.9, 9.1 9.6, 9.2 10.6
  //   E 256, 4 of 8 groups      8.8 6.2, 8.9 6.8, 9.3 8.1, 10.0 8.8, 10.4 10.8, 10.4 11.4, 10.7 12.3
  //   E 256, softmax, no bias   5.9 4.2, 6.0 4.6, 6.0 5.1, 6.3 5.6, 6.4 6.3, 6.5 7.0, 6.5 7.6
  // k + 2 experts have to fit 16 lanes.
  if (a.T >= (quarter_need <= 8 ? 4096 : 6144) && a.G <= 16 && quarter_need <= 16 && a.k <= 14 && a.k + a.S <= 16) {
    if (quarter_need <= 4) launch_quarter<4>(a, quarter_lanes, vec(4), s);
    else if (quarter_need <= 8) launch_quarter<8>(a, quarter_lanes, vec(8), s);
    else launch_quarter<16>(a, quarter_lanes, vec(16), s);
  } else if (need <= 1) launch_wave<1>(a, log2_lanes, vec(1), s);
  else if (need <= 2) launch_wave<2>(a, log2_lanes, vec(2), s);
  else if (need <= 4) launch_wave<4>(a, log2_lanes, vec(4), s);
  else if (need <= 8) launch_wave<8>(a, log2_lanes, vec(8), s);
  else {
    const int grid = a.T < (1 << 20) ? a.T : (1 << 20);
    hipLaunchKernelGGL(k_topk_lds, dim3(grid), dim3(64), (size_t)a.E * 8, s, a);
  }
  return hipGetLastError();
}

}  // namespace mm
