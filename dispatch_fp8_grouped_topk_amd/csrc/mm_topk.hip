// Choice of experts: scores, balance bias, expert groups, top-k and weights.
//
// One wave per row of logits.  Order is decided in float64, so that it does not depend on how an
// exponential is rounded: two scores that differ as real numbers compare as they do unless they lie
// within about 2^-50 of one another.  Without a bias the score is a monotone function of the logit and the
// logits themselves are compared.
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

__global__ __launch_bounds__(64) void k_topk(TopkArgs a) {
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

}  // namespace

hipError_t launch_gate_topk(const TopkArgs& a, hipStream_t s) {
  const int grid = a.T < (1 << 20) ? a.T : (1 << 20);
  hipLaunchKernelGGL(k_topk, dim3(grid), dim3(64), (size_t)a.E * 8, s, a);
  return hipGetLastError();
}

}  // namespace mm
