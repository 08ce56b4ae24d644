// Routing from logits: softmax or sigmoid scores, a balance bias that moves
// the choice but not the gates, expert groups, top-k, gates renormalised or as
// they are, a scale.
//
// For a row l of N logits (masked: NaN or -inf):
//   score   softmax p_e = exp(l_e - M) / sum, or sigmoid s_e = 1 / (1 + exp(-l_e))
//   value   c_e = l_e without a bias (both scores grow with the logit), else
//           score_e + b_e; NaN and -inf values are masked too
//   groups  G of N / G consecutive experts; a group is worth its largest value
//           or the sum of its two best scores (+ bias); the best ones are kept
//   choice  the k largest values of the kept groups, the lower index first on
//           equal values, masked experts last
//   gates   the scores of the chosen (0 for masked ones), over their sum when
//           renormalised, times the scale
// Which of two values is larger is decided as in 64 bits.
#pragma once
#include "common.cuh"

namespace bfmoe {

struct RouteCfg {
  int score, n_groups, top_groups, group_score, renorm;
  float scale;
};

__device__ __forceinline__ bool masked_logit(float l) { return !(l > -INFINITY); }

// Sum, maximum and best (value, index) over a warp; every lane gets the same.
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL_MASK, v, o));
  return v;
}
__device__ __forceinline__ void warp_best(double& v, int& i) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double ov = __shfl_xor_sync(FULL_MASK, v, o);
    const int oi = __shfl_xor_sync(FULL_MASK, i, o);
    if (ov > v || (ov == v && oi < i)) {
      v = ov;
      i = oi;
    }
  }
}

// The scores of one row in 64 bits.
struct Scores64 {
  float M;    // the largest logit (softmax)
  double Z;   // sum of exp(l - M)
  int score;
  __device__ __forceinline__ double unit(float l) const {
    return M == INFINITY ? (l == INFINITY ? 1.0 : 0.0) : exp(static_cast<double>(l) - static_cast<double>(M));
  }
  __device__ __forceinline__ double of(float l) const {
    if (score == BFMOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-static_cast<double>(l)));
    return unit(l) / Z;
  }
  // (l: not masked)
  __device__ __forceinline__ double value(float l, const float* bias, int e) const {
    return bias ? of(l) + static_cast<double>(bias[e]) : static_cast<double>(l);
  }
};

// Experts and gates of one row by one warp, everything in 64 bits.  Lane j
// ends with the expert of slot j.
template <typename Tl>
__device__ void route_row_64(const Tl* row, int N, int k, const RouteCfg& cfg, const float* __restrict__ bias, int lane,
                             int& e_out, float& gate_out) {
  Scores64 sc;
  sc.score = cfg.score;
  sc.M = 0.f;
  sc.Z = 1.0;
  if (cfg.score == BFMOE_SCORE_SOFTMAX) {
    float m = -INFINITY;
    for (int e = lane; e < N; e += 32) m = fmaxf(m, to_f32(row[e]));  // fmaxf drops NaN
    sc.M = warp_max(m);
    double z = 0.0;
    for (int e = lane; e < N; e += 32) {
      const float l = to_f32(row[e]);
      if (!masked_logit(l)) z += sc.unit(l);
    }
    sc.Z = warp_sum(z);
  }
  const int per = N / cfg.n_groups;
  unsigned long long kept = ~0ull;
  if (cfg.top_groups < cfg.n_groups) {
    // group values: lane g % 32 holds groups g and g + 32
    double gv[2] = {-INFINITY, -INFINITY};
    for (int g = 0; g < cfg.n_groups; ++g) {
      double a = -INFINITY, b = -INFINITY;  // the two best of the group
      for (int q = lane; q < per; q += 32) {
        const int e = g * per + q;
        const float l = to_f32(row[e]);
        if (masked_logit(l)) continue;
        double v = sc.value(l, bias, e);
        if (!(v > -INFINITY)) continue;
        if (cfg.group_score == BFMOE_GROUP_TOP2 && !bias) v = sc.of(l);
        if (v > a) {
          b = a;
          a = v;
        } else if (v > b) {
          b = v;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double oa = __shfl_xor_sync(FULL_MASK, a, o), ob = __shfl_xor_sync(FULL_MASK, b, o);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
      }
      if (cfg.group_score == BFMOE_GROUP_TOP2 && b > -INFINITY) a += b;
      if ((g & 31) == lane) gv[g >> 5] = a;
    }
    kept = 0ull;
    for (int q = 0; q < cfg.top_groups; ++q) {
      double v = -INFINITY;
      int i = 0x7fffffff;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int g = lane + 32 * h;
        if (g < cfg.n_groups && !((kept >> g) & 1ull) && (gv[h] > v || (gv[h] == v && g < i))) {
          v = gv[h];
          i = g;
        }
      }
      warp_best(v, i);
      kept |= 1ull << i;
    }
  }
  double pv = INFINITY;
  int pi = -1;
  int mine = 0;
  for (int j = 0; j < k; ++j) {
    double v = -INFINITY;
    int i = 0x7fffffff;
    for (int e = lane; e < N; e += 32) {
      if (!((kept >> (cfg.n_groups > 1 ? e / per : 0)) & 1ull)) continue;
      const float l = to_f32(row[e]);
      double c = masked_logit(l) ? -INFINITY : sc.value(l, bias, e);
      if (!(c > -INFINITY)) c = -INFINITY;
      if (!(c < pv || (c == pv && e > pi))) continue;  // ranks before the last pick
      if (c > v || (c == v && e < i)) {
        v = c;
        i = e;
      }
    }
    warp_best(v, i);
    pv = v;
    pi = i;
    if (lane == j) mine = i;
  }
  // gates: lane j < k
  float l = -INFINITY;
  bool live = false;
  if (lane < k) {
    l = to_f32(row[mine]);
    live = !masked_logit(l) && sc.value(l, bias, mine) > -INFINITY;
  }
  double u = 0.0;
  if (!cfg.renorm) {
    u = live ? sc.of(l) : 0.0;
  } else {
    const float m = warp_max(live ? l : -INFINITY);
    if (live) {
      if (cfg.score == BFMOE_SCORE_SOFTMAX) {
        u = m == INFINITY ? (l == INFINITY ? 1.0 : 0.0) : exp(static_cast<double>(l) - static_cast<double>(m));
      } else {
        // over exp(min(m, 0)), so that a row of very low logits keeps its ratios
        const double low = m < 0.f ? static_cast<double>(m) : 0.0;
        u = l > 0.f ? 1.0 / (1.0 + exp(-static_cast<double>(l)))
                    : exp(static_cast<double>(l) - low) / (1.0 + exp(static_cast<double>(l)));
      }
    }
    const double s = warp_sum(u);
    u = s > 0.0 ? u / s : 0.0;
  }
  e_out = mine;
  gate_out = static_cast<float>(u) * cfg.scale;
}

constexpr int kRouteWarps = 8;

template <typename Tl>
__global__ __launch_bounds__(kRouteWarps * 32) void route_kernel(const Tl* __restrict__ logits, long long ld, int T,
                                                                 int N, int k, RouteCfg cfg,
                                                                 const float* __restrict__ bias,
                                                                 int32_t* __restrict__ idx,
                                                                 float* __restrict__ gates) {
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * kRouteWarps;
  for (int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5); t < T; t += warps) {
    int e;
    float g;
    route_row_64(logits + static_cast<long long>(t) * ld, N, k, cfg, bias, lane, e, g);
    if (lane < k) {
      idx[static_cast<long long>(t) * k + lane] = e;
      gates[static_cast<long long>(t) * k + lane] = g;
    }
  }
}

}  // namespace bfmoe
