// Choice of experts: scores, balance bias, expert groups, top-k and weights.
//
// One wave per row of logits.  Order is decided in float64, so that it does not depend on how an
// exponential is rounded: two scores that differ as real numbers compare as they do unless they lie
// within about 2^-50 of one another.  Without a bias the score is a monotone function of the logit and the
// logits themselves are compared.
//
// k_topk_wave holds the row in registers, up to 16 experts a lane; k_topk_lds takes the rows that do not
// fit (more than 1024 experts, or groups that leave too few lanes each) through LDS.
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

// exp(x) in float64 to about an ulp, for any x (NaN excepted): x = n ln 2 + r with |r| <= ln 2 / 2, the
// Taylor series of exp(r) to r^13 / 13! (the next term is below 2^-57), times 2^n.
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

// The two largest of a group's values, group of 2^kLog neighbouring lanes (-inf where there is none).
__device__ __forceinline__ void best_two(double& m1, double& m2, int log2_lanes) {
  const auto merge = [&](double o1, double o2) {
    m2 = fmax(fmin(m1, o1), fmax(m2, o2));
    m1 = fmax(m1, o1);
  };
  if (log2_lanes >= 1) merge(dpp<kXor1>(m1), dpp<kXor1>(m2));
  if (log2_lanes >= 2) merge(dpp<kXor2>(m1), dpp<kXor2>(m2));
  if (log2_lanes >= 3) merge(dpp<kHalfMirror>(m1), dpp<kHalfMirror>(m2));
  if (log2_lanes >= 4) merge(dpp<kMirror>(m1), dpp<kMirror>(m2));
  if (log2_lanes >= 5) merge(__shfl_xor(m1, 16), __shfl_xor(m2, 16));
}

// kN experts a lane.  The lanes of a group are neighbours (2^log2_lanes of them), and experts go to lanes
// and places in ascending order, so that of equal values the lowest lane's lowest place is the lowest id.
// Each round takes the largest key of the wave: a DPP maximum, a ballot for the first lane that
// has it.  kBiased: keys are float64 values' (the lower halves are compared where the upper ones tie).
template <int kN, bool kBiased>
__global__ __launch_bounds__(256) void k_topk_wave(TopkArgs a, int log2_lanes, int vec) {
  const int lane = threadIdx.x & 63, cols = a.k + a.S, n = a.E / a.G;
  const int g = lane >> log2_lanes, i0 = (lane & ((1 << log2_lanes) - 1)) * kN;
  const int e0 = g * n + i0, mine = g < a.G ? min(max(n - i0, 0), kN) : 0;     // this lane's experts
  const bool need_scores = kBiased || (a.G > 1 && a.group_top == 2);
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
    float l[kN];
    const size_t at = (size_t)row * a.stride + e0;
    if (vec) {                                   // whole lanes, aligned
      if (a.bf16) {
        const uint16_t* p = static_cast<const uint16_t*>(a.logits) + at;
        uint16_t u[kN] = {};
        if (mine) __builtin_memcpy(u, __builtin_assume_aligned(p, kN * 2 < 16 ? kN * 2 : 16), kN * 2);
#pragma unroll
        for (int j = 0; j < kN; ++j) l[j] = __uint_as_float((uint32_t)u[j] << 16);
      } else {
        const float* p = static_cast<const float*>(a.logits) + at;
#pragma unroll
        for (int j = 0; j < kN; ++j) l[j] = 0.f;
        if (mine) __builtin_memcpy(l, __builtin_assume_aligned(p, kN * 4 < 16 ? kN * 4 : 16), kN * 4);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) l[j] = j < mine ? load_logit(a, at + j) : -kInf32;
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      l[j] = j < mine ? cleaned(l[j]) : -kInf32;
      if (l[j] > -kInf32) top = max(top, key32(l[j]));
    }
    // the softmax's largest logit; its sum where the scores themselves are asked for
    float lmax = 0.f;
    double total = 1.0;
    if (!a.sigmoid) {
      const uint32_t k = lane_value(wave_max63(top), 63);
      lmax = k ? value32(k) : 0.f;
      if (need_scores) {
        double t = 0.0;
#pragma unroll
        for (int j = 0; j < kN; ++j) t += l[j] == lmax ? 1.0 : exp64((double)l[j] - (double)lmax);
        total = lane_value(wave_sum63(t), 63);
      } else if (!a.renorm) {
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < kN; ++j) t += l[j] == lmax ? 1.f : __expf(l[j] - lmax);
        total = lane_value(wave_sum63((double)t), 63);
      }
      // renormalised without a bias: the sum cancels (the chosen ones hold at least 1/2048 of it, which
      // 1e-20 does not change)
    }
    const auto score = [&](float v) -> double {
      if (a.sigmoid) return 1.0 / (1.0 + exp64(-(double)v));
      return (v == lmax ? 1.0 : exp64((double)v - (double)lmax)) / total;
    };

    uint32_t hi[kN], lo[kN];
    double m1 = kNone, m2 = kNone;               // the lane's two largest ordering values
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const bool on = l[j] > -kInf32;
      hi[j] = lo[j] = 0;
      if constexpr (kBiased) {
        const float b = j < mine ? cleaned(a.bias[e0 + j]) : -kInf32;
        if (on && b > -kInf32) {
          const double c = score(l[j]) + (double)b;
          const uint64_t k = key64(c);
          hi[j] = (uint32_t)(k >> 32);
          lo[j] = (uint32_t)k;
          m2 = fmax(m2, fmin(m1, c));
          m1 = fmax(m1, c);
        }
      } else if (on) {
        hi[j] = key32(l[j]);
        m2 = fmax(m2, fmin(m1, (double)l[j]));
        m1 = fmax(m1, (double)l[j]);
      }
    }

    if (a.G > 1) {
      best_two(m1, m2, log2_lanes);
      double v = m1;
      if (a.group_top == 2 && m1 > kNone) {
        if constexpr (kBiased) v = m2 > kNone ? m1 + m2 : m1;
        else v = score((float)m1) + (m2 > kNone ? score((float)m2) : 0.0);
      }
      int rank = 0;                              // groups that come before this lane's
      for (int o = 0; o < a.G; ++o) {
        const double u = lane_value(v, o << log2_lanes);
        rank += u > v || (u == v && o < g);
      }
      if (rank >= a.KG) {
#pragma unroll
        for (int j = 0; j < kN; ++j) hi[j] = lo[j] = 0;
      }
    }

    int chosen = -1;                             // lane j: the j-th chosen expert and its logit
    float logit = 0.f;
    for (int r = 0; r < a.k; ++r) {
      uint32_t bh = hi[0], bl = lo[0];
      int bj = 0;
#pragma unroll
      for (int j = 1; j < kN; ++j) {
        const bool take = kBiased ? ((uint64_t)hi[j] << 32 | lo[j]) > ((uint64_t)bh << 32 | bl) : hi[j] > bh;
        bh = take ? hi[j] : bh;
        if constexpr (kBiased) bl = take ? lo[j] : bl;
        bj = take ? j : bj;
      }
      const uint32_t mh = lane_value(wave_max63(bh), 63);
      if (mh == 0) break;                        // nothing left to choose
      uint64_t who = __ballot(bh == mh);
      if constexpr (kBiased) {
        if (who & (who - 1)) {
          const uint32_t ml = lane_value(wave_max63(bh == mh ? bl : 0u), 63);
          who = __ballot(bh == mh && bl == ml);
        }
      }
      const int winner = __builtin_ctzll(who);
      const int j = __builtin_amdgcn_readlane(bj, winner);
      float lj = l[0];
#pragma unroll
      for (int q = 1; q < kN; ++q) lj = j == q ? l[q] : lj;
      const int e = __builtin_amdgcn_readlane(e0, winner) + j;
      const float v = __uint_as_float(lane_value(__float_as_uint(lj), winner));
      if (lane == r) {
        chosen = e;
        logit = v;
      }
#pragma unroll
      for (int q = 0; q < kN; ++q)
        if (lane == winner && q == j) hi[q] = lo[q] = 0;
    }
    double s = chosen >= 0 ? score(logit) : 0.0;
    if (a.renorm) s /= lane_value(wave_sum63(s), 63) + 1e-20;
    if (lane < a.k) {
      idx[lane] = chosen;
      w[lane] = (float)(s * (double)a.scale);
    } else if (lane < cols) {
      idx[lane] = a.E + lane - a.k;
      w[lane] = a.shared_weight;
    }
  }
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
  if (need <= 1) launch_wave<1>(a, log2_lanes, vec(1), s);
  else if (need <= 2) launch_wave<2>(a, log2_lanes, vec(2), s);
  else if (need <= 4) launch_wave<4>(a, log2_lanes, vec(4), s);
  else if (need <= 8) launch_wave<8>(a, log2_lanes, vec(8), s);
  else if (need <= 16) launch_wave<16>(a, log2_lanes, vec(16), s);
  else {
    const int grid = a.T < (1 << 20) ? a.T : (1 << 20);
    hipLaunchKernelGGL(k_topk_lds, dim3(grid), dim3(64), (size_t)a.E * 8, s, a);
  }
  return hipGetLastError();
}

}  // namespace mm
