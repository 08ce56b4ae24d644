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
__device__ __noinline__ void route_row_64(const Tl* row, int N, int k, const RouteCfg& cfg, const float* __restrict__ bias, int lane,
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

// exp(x) and 1 / x to about two units in the last place (plus |x| half steps
// for the argument of exp); results below the normal range become 0.
__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp(l - m), a maximum of +inf shared among the +inf logits (l not masked)
__device__ __forceinline__ float unit_softmax(float l, float m) {
  return m == INFINITY ? (l == INFINITY ? 1.f : 0.f) : exp_fast(l - m);
}
__device__ __forceinline__ float sigmoid_fast(float l) { return rcp_fast(1.f + exp_fast(-l)); }
// sigmoid(l) over exp(low), low = min(row maximum, 0): a row of very low
// logits keeps its ratios
__device__ __forceinline__ float unit_sigmoid(float l, float low) {
  return l > 0.f ? sigmoid_fast(l) : exp_fast(l - low) * rcp_fast(1.f + exp_fast(l));
}

// Unsigned integers in the order of the floats (no NaN).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o ^ ((o & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// Reductions over the LPR neighbouring lanes that share a row.
template <int LPR>
__device__ __forceinline__ uint32_t seg_max_u32(uint32_t v) {
  if constexpr (LPR == 32) {
    return __reduce_max_sync(FULL_MASK, v);
  } else {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(FULL_MASK, v, o));
    return v;
  }
}
template <int LPR>
__device__ __forceinline__ float seg_max(float v) {
  return from_ordered(seg_max_u32<LPR>(ordered(v)));
}
template <int LPR>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
  return v;
}
// Bits of the caller's row in a warp ballot, from bit 0.
template <int LPR>
__device__ __forceinline__ unsigned seg_bits(bool p, int lane) {
  const unsigned b = __ballot_sync(FULL_MASK, p);
  if constexpr (LPR == 32) return b;
  else return (b >> (lane & ~(LPR - 1))) & ((1u << LPR) - 1u);
}

// How a row of up to LPR * V logits lies in the registers of LPR lanes: in
// cells of CE consecutive experts, cell c of lane q holding experts
// (c * LPR + q) * CE ..., so that a lane's loads are wide and its neighbours'
// follow it.
template <int LPR_, int V_>
struct RowShape {
  static constexpr int LPR = LPR_, V = V_;
  static constexpr int CE = V < 8 ? V : 8;
  static constexpr int C = V / CE;
  static constexpr int IB = CE == 8 ? 3 : (CE == 4 ? 2 : 1);
  static constexpr int CB = C == 4 ? 2 : (C == 2 ? 1 : 0);
  static constexpr int ROWS = 32 / LPR;  // rows of a warp
  static constexpr int MAXN = LPR * V;
};

// Loads the lane's logits of a row: -inf for masked ones and behind the row's
// end.  wide: rows are
// whole cells of 16-byte (float32: 32-byte cells in two) aligned memory.
template <class S, typename Tl>
__device__ __forceinline__ void load_row(const Tl* row, int N, int q, bool wide, float (&l)[S::V]) {
#pragma unroll
  for (int c = 0; c < S::C; ++c) {
    const int e0 = (c * S::LPR + q) * S::CE;
    if (wide) {
      if (e0 < N) {
        if constexpr (sizeof(Tl) == 4) {
          static_assert(S::CE >= 4);
#pragma unroll
          for (int h = 0; h < S::CE; h += 4) {
            const float4 v = *reinterpret_cast<const float4*>(row + e0 + h);
            l[c * S::CE + h] = v.x;
            l[c * S::CE + h + 1] = v.y;
            l[c * S::CE + h + 2] = v.z;
            l[c * S::CE + h + 3] = v.w;
          }
        } else {
          uint32_t w[S::CE / 2];
          if constexpr (S::CE == 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + e0);
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(row + e0);
            w[0] = v.x;
            w[1] = v.y;
          }
#pragma unroll
          for (int h = 0; h < S::CE / 2; ++h) {
            l[c * S::CE + 2 * h] = __uint_as_float(w[h] << 16);
            l[c * S::CE + 2 * h + 1] = __uint_as_float(w[h] & 0xffff0000u);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < S::CE; ++i) l[c * S::CE + i] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < S::CE; ++i) l[c * S::CE + i] = e0 + i < N ? to_f32(row[e0 + i]) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < S::V; ++i) l[i] = fmaxf(l[i], -INFINITY);  // NaN becomes -inf
}
// Whether load_row may take its wide form for rows ld apart.
template <class S, typename Tl>
__host__ __device__ __forceinline__ bool wide_rows(const void* p, long long ld, int N) {
  return N % S::CE == 0 && ld % S::CE == 0 && (reinterpret_cast<uintptr_t>(p) & (S::CE * sizeof(Tl) - 1) & 15u) == 0;
}

// Scratch of the group values: a warp's rows, the values of one row.
__host__ __device__ constexpr size_t route_group_floats(int maxn) { return static_cast<size_t>(maxn); }

// A row in the registers of LPR lanes, N <= LPR * V.
//
// Ranking.  A value becomes a 32-bit key: its bits in integer order, the last
// B of them replaced by its place in the lane (the lower the expert, the
// larger), so that a lane's keys differ and its largest names its expert.  A
// pick is one warp-wide integer maximum of the lanes' largest keys without
// the place inside a cell; among equal ones the lowest lane has the lowest
// expert.  The lane that was picked finds its next key by one pass over its
// cell: max(key - picked) in wrapping arithmetic is the largest key below the
// picked one, and no key has to be moved.
// The truncated keys and the float32 scores rank two values rightly when they
// are further apart than both errors; k + 1 picks are taken and every gap is
// looked at.  The few rows (about 1 in 1000) with a smaller gap are settled in
// 64 bits by the whole warp (route_row_64).
// Values that the keys hold exactly (no bias: bfloat16 logits) need no gap.
template <class S, typename Tl>
__global__ __launch_bounds__(kRouteWarps * 32) void route_fast_kernel(const Tl* __restrict__ logits, long long ld,
                                                                      int T, int N, int k, RouteCfg cfg,
                                                                      const float* __restrict__ bias, bool wide,
                                                                      int lpg, int32_t* __restrict__ idx,
                                                                      float* __restrict__ gates) {
  constexpr int LPR = S::LPR, V = S::V, CE = S::CE, C = S::C;
  constexpr int B = S::IB + S::CB;
  constexpr uint32_t LOW = (1u << B) - 1u;
  extern __shared__ float route_smem[];  // bias [MAXN], then the group values
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int q = lane & (LPR - 1);
  const bool softmax = cfg.score == BFMOE_SCORE_SOFTMAX;
  const bool grouped = cfg.top_groups < cfg.n_groups;
  const bool top2 = grouped && cfg.group_score == BFMOE_GROUP_TOP2;
  const bool scored = bias || top2;
  const bool need_z = softmax && (scored || !cfg.renorm);
  const int per = N / cfg.n_groups;
  const bool cells = per % CE == 0;  // no cell lies in two groups
  float* gs = route_smem + S::MAXN + (w * S::ROWS + lane / LPR) * S::MAXN;
  if (bias) {
    for (int e = threadIdx.x; e < S::MAXN; e += blockDim.x) route_smem[e] = e < N ? bias[e] : 0.f;
    __syncthreads();
  }
  // float32 scores are off by less than this (times their size: the sum of a
  // softmax collects a half step a term at worst)
  const float eps_s = 0x1p-23f * (softmax ? 24.f + 0.5f * V : 4.f);
  const bool exact_keys = !bias && sizeof(Tl) == 2;

  const int warps = gridDim.x * kRouteWarps;
  for (int t0 = (blockIdx.x * kRouteWarps + w) * S::ROWS; t0 < T; t0 += warps * S::ROWS) {
    const int t = t0 + lane / LPR;
    const bool has = t < T;
    const Tl* row = logits + static_cast<long long>(has ? t : t0) * ld;
    float l[V], c[V];
    load_row<S>(row, N, q, wide, l);
    float m = 0.f, inv_z = 1.f;
    if (need_z) {
      float x = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) x = fmaxf(x, l[i]);
      m = seg_max<LPR>(x);
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        c[i] = masked_logit(l[i]) ? 0.f : unit_softmax(l[i], m);
        z += c[i];
      }
      z = seg_sum<LPR>(z);
      inv_z = z > 0.f ? 1.f / z : 0.f;
    }
    if (scored) {
#pragma unroll
      for (int cc = 0; cc < C; ++cc) {
        const int e0 = (cc * LPR + q) * CE;
        float b[CE];
#pragma unroll
        for (int h = 0; h < CE; h += 4) {
          const float4 v = bias ? *reinterpret_cast<const float4*>(route_smem + e0 + h) : make_float4(0.f, 0.f, 0.f, 0.f);
          b[h] = v.x;
          b[h + 1] = v.y;
          b[h + 2] = v.z;
          b[h + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < CE; ++i) {
          const int v = cc * CE + i;
          const float x = (softmax ? c[v] * inv_z : sigmoid_fast(l[v])) + b[i];
          c[v] = masked_logit(l[v]) ? -INFINITY : fmaxf(x, -INFINITY);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = l[i];
    }
    // groups: the two best of each cell (or every value) go to shared memory,
    // lpg lanes take a group
    bool clear = true;
    unsigned long long kept = ~0ull;
    if (grouped) {
      const int items = cells ? per / CE : per;  // of a group
      if (cells) {
#pragma unroll
        for (int cc = 0; cc < C; ++cc) {
          float a = -INFINITY, b = -INFINITY;
#pragma unroll
          for (int i = 0; i < CE; ++i) {
            const float x = c[cc * CE + i];
            b = fmaxf(b, fminf(a, x));
            a = fmaxf(a, x);
          }
          const int cell = cc * LPR + q;
          gs[2 * cell] = a;
          gs[2 * cell + 1] = b;
        }
      } else {
#pragma unroll
        for (int cc = 0; cc < C; ++cc)
#pragma unroll
          for (int i = 0; i < CE; ++i) gs[(cc * LPR + q) * CE + i] = c[cc * CE + i];
      }
      __syncwarp();
      constexpr int GH = BFMOE_MAX_GROUPS / LPR;  // groups of a lane, at most
      float gv[GH];
#pragma unroll
      for (int h = 0; h < GH; ++h) {
        const int g = q / lpg + h * LPR;
        float a = -INFINITY, b = -INFINITY;
        if (g < cfg.n_groups && (h == 0 || lpg == 1)) {
          for (int it = q % lpg; it < items; it += lpg) {
            float oa, ob = -INFINITY;
            if (cells) {
              oa = gs[2 * (g * items + it)];
              ob = gs[2 * (g * items + it) + 1];
            } else {
              oa = gs[g * items + it];
            }
            b = fmaxf(fminf(a, oa), fmaxf(b, ob));
            a = fmaxf(a, oa);
          }
        }
        if (h == 0)
          for (int o = 1; o < lpg; o <<= 1) {
            const float oa = __shfl_xor_sync(FULL_MASK, a, o), ob = __shfl_xor_sync(FULL_MASK, b, o);
            b = fmaxf(fminf(a, oa), fmaxf(b, ob));
            a = fmaxf(a, oa);
          }
        gv[h] = top2 && b > -INFINITY ? a + b : a;
      }
      int rank[GH];
#pragma unroll
      for (int h = 0; h < GH; ++h) rank[h] = 0;
#pragma unroll
      for (int h = 0; h < GH; ++h) {
        const int n = min(cfg.n_groups - h * LPR, LPR / lpg);
        for (int o = 0; o < n; ++o) {
          const float v = __shfl_sync(FULL_MASK, gv[h], (lane & ~(LPR - 1)) + o * lpg);
          const int g2 = o + h * LPR;
#pragma unroll
          for (int u = 0; u < GH; ++u) rank[u] += v > gv[u] || (v == gv[u] && g2 < q / lpg + u * LPR);
        }
      }
      float worst = INFINITY, best = -INFINITY;  // of the kept, of the others
      kept = 0ull;
#pragma unroll
      for (int h = 0; h < GH; ++h) {
        const int g = q / lpg + h * LPR;
        const bool real = g < cfg.n_groups && (h == 0 || lpg == 1) && q % lpg == 0;
        const bool in = real && rank[h] < cfg.top_groups;
        if (in) worst = fminf(worst, gv[h]);
        else if (real) best = fmaxf(best, gv[h]);
        // bit g * lpg of the ballot; moved to bit g below by the reader
        kept |= static_cast<unsigned long long>(seg_bits<LPR>(in, lane)) << (h * LPR);
      }
      if (scored) {
        worst = -seg_max<LPR>(-worst);
        best = seg_max<LPR>(best);
        // (a sum of two scores; the score itself is at most 1)
        const float e = 4.f * (eps_s + 0x1p-23f * (1.f + fabsf(worst)));
        clear = !(best > -INFINITY) || worst - best > e;
      }
      if (scored && !bias) {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = l[i];
      }
    }
    // keys: 0 what is no candidate, then masked experts, then values
    uint32_t key[V];
#pragma unroll
    for (int cc = 0; cc < C; ++cc) {
      const int e0 = (cc * LPR + q) * CE;
      int g = 0, r = 0;
      bool in = true;
      if (grouped) {
        g = e0 / per;
        r = e0 - g * per;
        in = (kept >> (g * lpg)) & 1ull;
      }
#pragma unroll
      for (int i = 0; i < CE; ++i) {
        const uint32_t low = static_cast<uint32_t>((C - 1 - cc) * CE + (CE - 1 - i));
        const float x = c[cc * CE + i];
        const uint32_t o = x > -INFINITY ? (ordered(x + 0.f) & ~LOW) | low : (1u << B) | low;  // + 0: one zero
        if (grouped && !cells) {
          if (r == per) {
            r = 0;
            ++g;
            in = (kept >> (g * lpg)) & 1ull;
          }
          ++r;
        }
        key[cc * CE + i] = in && e0 + i < N ? o : 0u;
      }
    }
    uint32_t head[C];
#pragma unroll
    for (int cc = 0; cc < C; ++cc) {
      head[cc] = key[cc * CE];
#pragma unroll
      for (int i = 1; i < CE; ++i) head[cc] = max(head[cc], key[cc * CE + i]);
    }
    // picks: lane j of the row keeps the j-th (key and lane)
    uint32_t pick = 0;
    int from = 0;
    for (int j = 0; j <= k; ++j) {
      uint32_t top = head[0];
#pragma unroll
      for (int cc = 1; cc < C; ++cc) top = max(top, head[cc]);
      const uint32_t best = seg_max_u32<LPR>(top >> S::IB);
      const unsigned who = seg_bits<LPR>((top >> S::IB) == best, lane);
      const int src = __ffs(who) - 1;
      const uint32_t got = __shfl_sync(FULL_MASK, top, src, LPR);
      if (q == j) {
        pick = got;
        from = src;
      }
      if (q == src) {
        const int cc = C - 1 - static_cast<int>((got & LOW) >> S::IB);
#pragma unroll
        for (int u = 0; u < C; ++u)
          if (u == cc) {
            uint32_t d = 0u - got;
#pragma unroll
            for (int i = 0; i < CE; ++i) d = max(d, key[u * CE + i] - got);
            head[u] = got + d;
          }
      }
    }
    // the picks' values again, the gaps between them, the gates
    const bool valid = pick != 0u && q <= k;
    const int place = static_cast<int>(LOW) - static_cast<int>(pick & LOW);  // c * CE + i
    const int e = ((place / CE) * LPR + from) * CE + place % CE;
    const bool live = valid && (pick >> B) > 1u;
    float le = -INFINITY, sc = 0.f, val = 0.f, eps = 0.f;
    if (live) {
      le = to_f32(row[e]);
      if (scored || !cfg.renorm) sc = softmax ? unit_softmax(le, m) * inv_z : sigmoid_fast(le);
      val = bias ? sc + route_smem[e] : le;
      if (bias) eps = 0x1p-23f + eps_s * (softmax ? sc : 1.f) + 0x1p-23f * fabsf(val);
      if (!exact_keys) eps += fabsf(val) * (0x1p-23f * (1u << B)) + 0x1p-126f;
    }
    if (!exact_keys) {
      const float v2 = __shfl_down_sync(FULL_MASK, val, 1, LPR);
      const float e2 = __shfl_down_sync(FULL_MASK, eps, 1, LPR);
      const bool l2 = __shfl_down_sync(FULL_MASK, live ? 1 : 0, 1, LPR) != 0;
      const bool near = q < k && l2 && !(val - v2 > eps + e2);
      const unsigned nears = seg_bits<LPR>(near, lane);  // by every lane, whatever its row's groups said
      clear = clear && nears == 0u;
    }
    const bool mine = q < k && live;
    float u = 0.f;
    if (cfg.renorm) {
      const float top = seg_max<LPR>(mine ? le : -INFINITY);
      if (mine) u = softmax ? unit_softmax(le, top) : unit_sigmoid(le, fminf(top, 0.f));
      const float sum = seg_sum<LPR>(u);
      u = sum > 0.f ? u / sum : 0.f;
    } else if (mine) {
      u = sc;
    }
    if (has && clear && q < k) {
      idx[static_cast<long long>(t) * k + q] = e;
      gates[static_cast<long long>(t) * k + q] = u * cfg.scale;
    }
    unsigned open = __ballot_sync(FULL_MASK, has && !clear && q == 0);
    while (open) {
      const int t2 = t0 + (__ffs(open) - 1) / LPR;
      open &= open - 1;
      int e2;
      float g2;
      route_row_64(logits + static_cast<long long>(t2) * ld, N, k, cfg, bias, lane, e2, g2);
      if (lane < k) {
        idx[static_cast<long long>(t2) * k + lane] = e2;
        gates[static_cast<long long>(t2) * k + lane] = g2;
      }
    }
    if (grouped) __syncwarp();  // the group values are read before the next row's are written
  }
}

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
