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
#include <algorithm>

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

// exp(x) and 1 / x to about two units in the last place (plus |x| half steps
// for the argument of exp); results below the normal range become 0.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp_fast(float x) { return exp2_fast(x * 1.4426950408889634f); }
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

// A matrix of logits.  (The type is a template parameter all the way down: a
// test of it inside unrolled loops is predicated, and both sides are issued.)
template <typename T>
struct Logits {
  static constexpr bool BF16 = sizeof(T) == 2;
  const T* p;
  long long ld;
  int wide;  // rows are whole cells of memory aligned to cells (RowShape)
  __device__ __forceinline__ float at(int t, int e) const { return to_f32(p[static_cast<long long>(t) * ld + e]); }
};

// The score of a logit that is not masked, in 64 bits: M and Z the row's
// largest logit and sum of exp(l - M) (Z = 1: that term itself).  Rows that
// need it are few and their code is not in the instruction cache: one instance
// for all of them.
__device__ __noinline__ double score_64(float l, float M, double Z, bool softmax) {
  if (softmax && M == INFINITY) return (l == INFINITY ? 1.0 : 0.0) / Z;
  const double x = exp(softmax ? static_cast<double>(l) - static_cast<double>(M) : -static_cast<double>(l));
  return softmax ? x / Z : 1.0 / (1.0 + x);
}

// Float32 scores are off by less than this times their size: softmax, in half
// steps, 2.5 for each unit of the exponent (|x| p <= 0.37, and 17 on average
// over the sum: |x| <= ln N), 7 of the functions and products, one for each
// addition of the sum at worst, 16 for the rounding of m log2 e where |m| < 16 is
// folded into the exponents (row_softmax) ...
__device__ __forceinline__ float score_eps(bool softmax, int terms) {
  return 0x1p-23f * (softmax ? 32.f + 0.5f * static_cast<float>(terms) : 4.f);
}
// ... and a value by its score's error and its own rounding.
__device__ __forceinline__ float value_eps(float eps_s, bool softmax, float score, float value) {
  return 0x1p-23f + eps_s * (softmax ? score : 1.f) + 0x1p-23f * fabsf(value);
}

// A group's worth from its two best values.  A sum that leaves float32 at the
// lower end (two biases of the lowest value) is not that of an empty group.
__device__ __forceinline__ float group_worth(float a, float b, bool top2) {
  return top2 && b > -INFINITY ? fmaxf(a + b, -0x1.fffffep127f) : a;
}
// The bounds of a group's worth gv, the larger or the sum of the values a and b:
// their errors go by their own sizes, which the sum of a positive and a negative
// one does not show.
__device__ __forceinline__ float group_eps(float eps_s, bool softmax, float a, float b) {
  return 2.f * value_eps(eps_s, softmax, 1.f, fabsf(a) + (b > -INFINITY ? fabsf(b) : 0.f));
}
__device__ __forceinline__ float at_least(float gv, float eps) { return fabsf(gv) < INFINITY ? gv - eps : gv; }
__device__ __forceinline__ float at_most(float gv, float eps) { return fabsf(gv) < INFINITY ? gv + eps : gv; }

constexpr int kRouteWindow = 32;

// Experts and gates of row t by one warp, decided in 64 bits: groups from
// 64-bit values; the k best float32 values, which are the answer where values
// are logits; else every expert whose float32 value comes within its error of
// the k-th is ranked again by its 64-bit value (win: kRouteWindow ints of the
// warp's shared memory; more than that many: k passes over the whole row).
// Lane j ends with the expert of slot j.
template <typename Tl>
__device__ __noinline__ void route_row_64(const Logits<Tl>& x, int t, int N, int k, const RouteCfg& cfg,
                                          const float* __restrict__ bias, int* win, int lane, int& e_out,
                                          float& gate_out) {
  const bool softmax = cfg.score == BFMOE_SCORE_SOFTMAX;
  const bool grouped = cfg.top_groups < cfg.n_groups;
  const bool top2 = grouped && cfg.group_score == BFMOE_GROUP_TOP2;
  float M = 0.f;
  double Z = 1.0;
  if (softmax && (bias || top2 || !cfg.renorm)) {
    float m = -INFINITY;
    for (int e = lane; e < N; e += 32) m = fmaxf(m, x.at(t, e));  // fmaxf drops NaN
    M = warp_max(m);
    double z = 0.0;
#pragma unroll 1
    for (int e = lane; e < N; e += 32) {
      const float l = x.at(t, e);
      if (!masked_logit(l)) z += score_64(l, M, 1.0, true);
    }
    Z = warp_sum(z);
  }
  // -inf: masked
  auto value64 = [&](int e, bool score) {
    const float l = x.at(t, e);
    double v = -INFINITY;
    if (!masked_logit(l)) v = bias || score ? score_64(l, M, Z, softmax) : static_cast<double>(l);
    if (bias) v += static_cast<double>(bias[e]);
    return v > -INFINITY ? v : -INFINITY;  // NaN
  };
  const int per = N / cfg.n_groups;
  unsigned long long kept = ~0ull;
  if (grouped) {
    // group values: lane g % 32 holds groups g and g + 32
    double gv[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
    for (int g = 0; g < cfg.n_groups; ++g) {
      double a = -INFINITY, b = -INFINITY;  // the two best of the group
#pragma unroll 1
      for (int q = lane; q < per; q += 32) {
        const double v = value64(g * per + q, top2);
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
      if (top2 && b > -INFINITY) a += b;
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
  auto candidate = [&](int e) { return !grouped || ((kept >> (e / per)) & 1ull); };
  const float inv_z = softmax ? static_cast<float>(1.0 / Z) : 1.f;
  auto score32 = [&](float l) { return softmax ? unit_softmax(l, M) * inv_z : sigmoid_fast(l); };
  auto value32 = [&](int e) {  // -inf: masked
    const float l = x.at(t, e);
    if (masked_logit(l)) return -INFINITY;
    return bias ? fmaxf(score32(l) + bias[e], -INFINITY) : l;
  };
  int mine = 0;
  // the k best in float32
  float pv = INFINITY;
  int pi = -1;
  for (int j = 0; j < k; ++j) {
    float v = -INFINITY;
    int i = 0x7fffffff;
    for (int e = lane; e < N; e += 32) {
      if (!candidate(e)) continue;
      const float c = value32(e);
      if (!(c < pv || (c == pv && e > pi))) continue;  // ranks before the last pick
      if (c > v || (c == v && e < i)) {
        v = c;
        i = e;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ov = __shfl_xor_sync(FULL_MASK, v, o);
      const int oi = __shfl_xor_sync(FULL_MASK, i, o);
      if (ov > v || (ov == v && oi < i)) {
        v = ov;
        i = oi;
      }
    }
    pv = v;
    pi = i;
    if (lane == j) mine = i;
  }
  if (bias && pv < INFINITY) {
    const float eps_s = score_eps(softmax, N / 32);
    // (fewer than k experts left: everything is looked at)
    const float near = pv > -INFINITY ? pv - 2.f * value_eps(eps_s, softmax, 1.f, pv) : -INFINITY;
    int n = 0;
    __syncwarp();
    for (int e0 = 0; e0 < N; e0 += 32) {
      const int e = e0 + lane;
      const bool in = e < N && candidate(e) && value32(e) >= near;
      const unsigned b = __ballot_sync(FULL_MASK, in);
      const int at = n + __popc(b & ((1u << lane) - 1u));
      if (in && at < kRouteWindow) win[at] = e;
      n += __popc(b);
    }
    __syncwarp();
    if (n <= kRouteWindow) {
      double v = -INFINITY;
      int e = 0x7fffffff;
      if (lane < n) {
        e = win[lane];
        v = value64(e, false);
      }
      int rank = 0;
      for (int o = 0; o < n; ++o) {
        const double ov = __shfl_sync(FULL_MASK, v, o);
        const int oe = __shfl_sync(FULL_MASK, e, o);
        rank += ov > v || (ov == v && oe < e);
      }
      __syncwarp();
      if (lane < n) win[rank] = e;
      __syncwarp();
      if (lane < k) mine = win[lane];
      __syncwarp();
    } else {
      double pv64 = INFINITY;
      pi = -1;
      for (int j = 0; j < k; ++j) {
        double v = -INFINITY;
        int i = 0x7fffffff;
        for (int e = lane; e < N; e += 32) {
          if (!candidate(e)) continue;
          const double c = value64(e, false);
          if (!(c < pv64 || (c == pv64 && e > pi))) continue;
          if (c > v || (c == v && e < i)) {
            v = c;
            i = e;
          }
        }
        warp_best(v, i);
        pv64 = v;
        pi = i;
        if (lane == j) mine = i;
      }
    }
  }
  // gates: lane j < k
  float l = -INFINITY;
  bool live = false;
  if (lane < k) {
    l = x.at(t, mine);
    live = value32(mine) > -INFINITY;
  }
  float u = 0.f;
  if (cfg.renorm) {
    const float top = warp_max(live ? l : -INFINITY);
    if (live) u = softmax ? unit_softmax(l, top) : unit_sigmoid(l, fminf(top, 0.f));
    const float sum = warp_sum(u);
    u = sum > 0.f ? u / sum : 0.f;
  } else if (live) {
    u = score32(l);
  }
  e_out = mine;
  gate_out = u * cfg.scale;
}

constexpr int kRouteWarps = 8;

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
  static constexpr int ROWS = 32 / LPR;  // rows of a warp
  static constexpr int MAXN = LPR * V;
  static_assert(CE >= 2 && C <= 4);
};

// Where expert e's float32 lies in an array in shared memory that lanes read in
// cells: the halves of eight-expert cells apart, so that the 16 bytes of
// neighbouring lanes follow each other (32 apart, every read took two passes).
template <class S>
__device__ __forceinline__ int slot_of(int e) {
  if constexpr (S::CE < 8) return e;
  const int cell = e >> 3;
  return ((cell / S::LPR * 2 + ((e >> 2) & 1)) * S::LPR + cell % S::LPR) * 4 + (e & 3);
}
// A lane's cells of such an array.
template <class S>
__device__ __forceinline__ void load_cells(const float* a, int q, float (&v)[S::V]) {
  if constexpr (S::CE == 2) {
    const float2 f = *reinterpret_cast<const float2*>(a + q * 2);
    v[0] = f.x, v[1] = f.y;
  } else {
#pragma unroll
    for (int h = 0; h < S::V; h += 4) {
      const float4 f = *reinterpret_cast<const float4*>(a + (h / 4 * S::LPR + q) * 4);
      v[h] = f.x, v[h + 1] = f.y, v[h + 2] = f.z, v[h + 3] = f.w;
    }
  }
}

// Cell c of them, read and written.
template <class S>
__device__ __forceinline__ void load_cell_of(const float* a, int q, int c, float (&v)[S::CE]) {
#pragma unroll
  for (int h = 0; h < S::CE; h += 4) {
    const float4 f = *reinterpret_cast<const float4*>(a + ((c * S::CE + h) / 4 * S::LPR + q) * 4);
    v[h] = f.x, v[h + 1] = f.y, v[h + 2] = f.z, v[h + 3] = f.w;
  }
}
template <class S>
__device__ __forceinline__ void store_cell_of(float* a, int q, int c, const float (&v)[S::CE]) {
#pragma unroll
  for (int h = 0; h < S::CE; h += 4)
    *reinterpret_cast<float4*>(a + ((c * S::CE + h) / 4 * S::LPR + q) * 4) = make_float4(v[h], v[h + 1], v[h + 2], v[h + 3]);
}

// A row's words as they are in memory, so that the next row can be on its way
// while one is worked on.  Words behind the row's end are -inf of its type.
template <class S, typename Tl>
struct RawRow {
  static constexpr bool BF16 = sizeof(Tl) == 2;
  static constexpr int CW = S::CE * static_cast<int>(sizeof(Tl)) / 4;  // words of a cell: 1, 2, 4 or 8
  uint32_t w[S::V];

  // A cell from aligned memory (to its size), global or shared.
  template <bool GLOBAL>
  __device__ __forceinline__ void load_cell(int c, const Tl* p, bool in) {
    constexpr uint32_t M = BF16 ? 0xff80ff80u : 0xff800000u;
    if constexpr (CW == 8 && GLOBAL) {
      uint32_t* v = w + 8 * c;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = M;
      if (in)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "l"(p)
                     : "memory");
      return;
    }
    if constexpr (CW == 1) {
      w[c] = in ? *reinterpret_cast<const uint32_t*>(p) : M;
    } else if constexpr (CW == 2) {
      const uint2 u = in ? *reinterpret_cast<const uint2*>(p) : make_uint2(M, M);
      w[2 * c] = u.x, w[2 * c + 1] = u.y;
    } else {
#pragma unroll
      for (int h = 0; h < CW / 4; ++h) {
        const uint4 u = in ? reinterpret_cast<const uint4*>(p)[h] : make_uint4(M, M, M, M);
        w[CW * c + 4 * h] = u.x, w[CW * c + 4 * h + 1] = u.y;
        w[CW * c + 4 * h + 2] = u.z, w[CW * c + 4 * h + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void load(const Logits<Tl>& x, int t, int N, int q) {
    const Tl* row = x.p + static_cast<long long>(t) * x.ld;
    if (x.wide) {
#pragma unroll
      for (int c = 0; c < S::C; ++c) {
        const int e0 = (c * S::LPR + q) * S::CE;
        load_cell<true>(c, row + e0, e0 < N);
      }
    } else {  // logit i is that of expert i LPR + q
#pragma unroll
      for (int i = 0; i < S::V; ++i) {
        const int e = i * S::LPR + q;
        if constexpr (BF16) w[i] = e < N ? reinterpret_cast<const uint16_t*>(row)[e] : 0xff80u;
        else w[i] = e < N ? reinterpret_cast<const uint32_t*>(row)[e] : 0xff800000u;
      }
    }
  }
  // The same words from a copy of the row in shared memory (all MAXN of it).
  __device__ __forceinline__ void load_shared(const uint8_t* row, int q) {
#pragma unroll
    for (int c = 0; c < S::C; ++c)
      load_cell<false>(c, reinterpret_cast<const Tl*>(row) + (c * S::LPR + q) * S::CE, true);
  }
  // The logits; FIX: NaN as -inf.
  template <bool FIX>
  __device__ __forceinline__ void unpack(bool wide, float (&l)[S::V]) const {
    if constexpr (BF16) {
      if (wide) {
#pragma unroll
        for (int i = 0; i < S::V / 2; ++i) {
          l[2 * i] = __uint_as_float(w[i] << 16);
          l[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < S::V; ++i) l[i] = __uint_as_float(w[i] << 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < S::V; ++i) l[i] = __uint_as_float(w[i]);
    }
    if constexpr (FIX) {
#pragma unroll
      for (int i = 0; i < S::V; ++i) l[i] = fmaxf(l[i], -INFINITY);
    }
  }
};
// Whether rows can be read in cells (Logits::wide).
template <class S, typename Tl>
inline bool wide_rows(const Tl* p, long long ld, int N) {
  const size_t bytes = S::CE * sizeof(Tl);
  return N % S::CE == 0 && ld % S::CE == 0 && reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

// Rows of more than 256 experts come through shared memory: one bulk copy a
// row, a row of each warp on its way while one is worked on.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// A warp's rows t0, t0 + step, ..., loads ahead of the work: rows of up to 256
// experts as registers, longer ones (in cells) through two buffers of the warp
// in shared memory.
template <class S, typename Tl>
struct RowFeed {
  static constexpr bool AHEAD = S::V <= 8;
  static constexpr int ROW = S::MAXN * static_cast<int>(sizeof(Tl));
  // Bytes of shared memory of a warp: rows in cells go through two buffers (not
  // AHEAD), others are brought into cells through one in float32.
  __host__ __device__ static constexpr int bytes(bool wide) { return wide ? (AHEAD ? 0 : 2 * S::ROWS * ROW) : S::ROWS * S::MAXN * 4; }
  RawRow<S, Tl> raw;
  uint8_t* buf;
  uint64_t* full;
  const uint8_t* here;  // the row in shared memory, or NULL
  int turn;
  bool staged;

  // one lane: the rows from t on into buffer b
  __device__ __forceinline__ void fetch(const Logits<Tl>& x, int t, int T, int N, int b) {
    const int bytes = N * static_cast<int>(sizeof(Tl)), rows = min(S::ROWS, T - t);
    mbar_expect_tx(full + b, rows * bytes);
    for (int r = 0; r < rows; ++r)
      bulk_load(buf + (b * S::ROWS + r) * ROW, x.p + static_cast<long long>(t + r) * x.ld, bytes, full + b);
  }
  // bars: two of the warp's (not AHEAD)
  __device__ __forceinline__ void start(const Logits<Tl>& x, int t0, int T, int N, int lane, uint8_t* buffer, uint64_t* bars) {
    here = nullptr;
    turn = 0;
    staged = !AHEAD && x.wide;
    buf = buffer;
    full = bars;
    if constexpr (AHEAD) {
      if (t0 < T) raw.load(x, min(t0 + lane / S::LPR, T - 1), N, lane & (S::LPR - 1));
    } else if (staged) {
      // behind the row's end the buffers hold -inf, which no copy reaches
      for (int e = N + lane; e < S::MAXN; e += 32)
        for (int b = 0; b < 2 * S::ROWS; ++b) reinterpret_cast<Tl*>(buf + b * ROW)[e] = from_f32<Tl>(-INFINITY);
      if (lane == 0) {
        mbar_init(full, 1);
        mbar_init(full + 1, 1);
        mbar_fence_init();
        if (t0 < T) fetch(x, t0, T, N, 0);
      }
      __syncwarp();
    }
  }
  // The logits of the warp's rows at t0 (past the end: anything).
  // False after a copy that did not come, which is reported: then nothing of
  // the warp's is on its way any more.
  template <bool FIX = true>
  __device__ __forceinline__ bool take(const Logits<Tl>& x, int t0, int step, int T, int N, int lane, float (&l)[S::V]) {
    const int q = lane & (S::LPR - 1);
    if constexpr (AHEAD) {
      raw.template unpack<FIX>(x.wide, l);
      if (t0 + step < T) raw.load(x, min(t0 + step + lane / S::LPR, T - 1), N, q);
    } else {
      if (staged) {
        const int b = turn & 1;
        // the buffer of the row before was read before that row's work
        if (lane == 0 && t0 + step < T) fetch(x, t0 + step, T, N, b ^ 1);
        if (__any_sync(FULL_MASK, !mbar_wait(full + b, (turn >> 1) & 1, 0x2100u))) {
          if (t0 + step < T) mbar_wait(full + (b ^ 1), ((turn + 1) >> 1) & 1, 0x2101u);
          return false;
        }
        here = buf + (b * S::ROWS + lane / S::LPR) * ROW;
        raw.load_shared(here, q);
        __syncwarp();
        ++turn;
      } else {
        raw.load(x, min(t0 + lane / S::LPR, T - 1), N, q);
      }
      raw.template unpack<FIX>(x.wide, l);
    }
    if (!x.wide) {
      float* cells = reinterpret_cast<float*>(buf) + lane / S::LPR * S::MAXN;
#pragma unroll
      for (int i = 0; i < S::V; ++i) cells[slot_of<S>(i * S::LPR + q)] = l[i];
      __syncwarp();
      load_cells<S>(cells, q, l);
      __syncwarp();
    }
    return true;
  }
  // After the rows at t0 were taken, for a warp that takes no more: the copy on
  // its way is waited for.
  __device__ __forceinline__ void drain(int t0, int step, int T) {
    if constexpr (!AHEAD) {
      if (staged && t0 + step < T) mbar_wait(full + (turn & 1), (turn >> 1) & 1, 0x2102u);
    }
  }
  // The row taken last once more (rows of registers are there still).
  __device__ __forceinline__ void again(const Logits<Tl>& x, int t, int N, int lane, float (&l)[S::V]) {
    if constexpr (!AHEAD) {
      if (here) {
        raw.load_shared(here, lane & (S::LPR - 1));
        raw.template unpack<true>(x.wide, l);
      } else {
        load_cells<S>(reinterpret_cast<const float*>(buf) + lane / S::LPR * S::MAXN, lane & (S::LPR - 1), l);
      }
    }
  }
  // Logit e of row t, the row taken last.
  __device__ __forceinline__ float at(const Logits<Tl>& x, int t, int e) const {
    return !AHEAD && here ? to_f32(reinterpret_cast<const Tl*>(here)[e]) : x.at(t, e);
  }
};

// Values i and i + 1 of a lane (two float32 operations an instruction), and the
// sum of all.
__device__ __forceinline__ float2 pair(const float* v, int i) { return make_float2(v[i], v[i + 1]); }
template <int V>
__device__ __forceinline__ float lane_sum(const float (&v)[V]) {
  float2 s = pair(v, 0);
#pragma unroll
  for (int i = 2; i < V; i += 2) s = __fadd2_rn(s, pair(v, i));
  return s.x + s.y;
}

// exp(l - m) of a row and its sum over the row; masked logits give 0.
template <class S>
__device__ __forceinline__ float row_softmax(const float (&l)[S::V], float m, float (&u)[S::V]) {
  if (fabsf(m) < 16.f) {
    const float2 by = make_float2(1.4426950408889634f, 1.4426950408889634f);
    const float2 ml = make_float2(-m * by.x, -m * by.x);
#pragma unroll
    for (int i = 0; i < S::V; i += 2) {
      const float2 x = __ffma2_rn(pair(l, i), by, ml);
      u[i] = exp2_fast(x.x);
      u[i + 1] = exp2_fast(x.y);
    }
  } else if (fabsf(m) < 0x1p120f) {
#pragma unroll
    for (int i = 0; i < S::V; ++i) u[i] = exp_fast(l[i] - m);
  } else {  // +-inf, or masks of the type's lowest value alone
#pragma unroll
    for (int i = 0; i < S::V; ++i) u[i] = masked_logit(l[i]) ? 0.f : unit_softmax(l[i], m);
  }
  return seg_sum<S::LPR>(lane_sum(u));
}

template <class S>
__device__ __forceinline__ float row_max(const float (&l)[S::V]) {
  float h = -INFINITY;
#pragma unroll
  for (int i = 0; i < S::V; ++i) h = fmaxf(h, l[i]);  // drops NaN
  return seg_max<S::LPR>(h);
}
// What ranks the experts: the logits, or softmax or sigmoid scores (with a
// bias, or summed up by group).
enum { kByLogit = 0, kBySoftmax = 1, kBySigmoid = 2 };

// Blocks of an SM.  (16384 x 256 in groups, with buckets: 30.4 us with 3 blocks
// of 80 registers a thread, 33.0 with 4 of 64.)
template <class S>
constexpr int kRouteBlocks = 3;

// Floats of shared memory for the group values of a row: all values in 64 bits
// where there is room for them.
template <class S>
constexpr int kGroupSpace = S::V <= 8 ? 2 * S::MAXN : S::MAXN;

// A candidate of a row.
struct Candidate {
  float value;
  int e;
  float eps;  // error of the value
  int pad;
};

// A warp a row, the row in its registers (N <= 32 V).
//
// Choice.  The (k + 1)-th largest of the lanes' maxima is at most the
// (k + 1)-th largest value of the row, and few values reach it (about 10 of
// 256 or 1024 for k = 8): those are the candidates, one a lane, ranked among
// each other by value and index.  (Picking the largest k + 1 times instead,
// with every value made into a sortable key, took 174 us for 131072 rows of
// 1024 experts, k = 4; this takes 107: 5.1 TB/s, bound by the instructions
// issued, about 500 a row.)
// Rows with more than 32 candidates (many equal values) are left for the end,
// to route_row_64.
//
// Scores are float32 and rank two values rightly only where they are further
// apart than their errors.  The threshold is lowered by both, and where two
// candidates are nearer (about 1 row in 1000) they are ranked by 64-bit values.
// Groups that are too near each other are treated alike.
template <class S, typename Tl, int BY, bool GROUPED>
__global__ __launch_bounds__(kRouteWarps * 32, kRouteBlocks<S>) void route_fast_kernel(
    const Logits<Tl> x, int T, int N, int k, const RouteCfg cfg, const float* __restrict__ bias, int lsh,
    int32_t* idx, float* __restrict__ gates) {
  constexpr int LPR = 32, V = S::V, CE = S::CE, C = S::C;
  static_assert(S::LPR == 32);
  constexpr bool SCORED = BY != kByLogit;
  extern __shared__ __align__(128) float route_smem[];  // bias [MAXN] (scored), group values (grouped), rows
  __shared__ Candidate cand_s[kRouteWarps][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, q = lane;
  const bool softmax = BY == kBySoftmax || (BY == kByLogit && cfg.score == BFMOE_SCORE_SOFTMAX);
  const int per = GROUPED ? N / cfg.n_groups : N;
  const bool cells = per % CE == 0;  // no cell lies in two groups
  float* gs = route_smem + (SCORED ? S::MAXN : 0) + w * kGroupSpace<S>;
  Candidate* cand = cand_s[w];
  pdl_wait();
  pdl_trigger();
  if constexpr (SCORED) {
    for (int e = threadIdx.x; e < S::MAXN; e += blockDim.x)
      route_smem[slot_of<S>(e)] = bias && e < N ? fmaxf(bias[e], -INFINITY) : 0.f;  // NaN masks
    __syncthreads();
  }
  const float eps_s = score_eps(softmax, V);
  // groups: 1 << lsh lanes take one; lane q works on group gq (+ 32, ...),
  // its cells begin in groups g0
  const int lpg = 1 << lsh, gq = q >> lsh;
  int g0[C];
  if constexpr (GROUPED) {
#pragma unroll
    for (int cc = 0; cc < C; ++cc) g0[cc] = (cc * LPR + q) * CE / per;
  }
  const int items = cells ? per / CE : per;  // of a group
  const bool by_lanes = GROUPED && C == 1 && cells && items == lpg;
  const bool top2 = cfg.group_score == BFMOE_GROUP_TOP2;
  const bool fits_64 = cells || kGroupSpace<S> >= 2 * S::MAXN;

  const int step = gridDim.x * kRouteWarps;
  int t = blockIdx.x * kRouteWarps + w;
  __shared__ uint64_t full_s[kRouteWarps * 2];
  RowFeed<S, Tl> feed;
  feed.start(x, t, T, N, lane,
             reinterpret_cast<uint8_t*>(route_smem + (SCORED ? S::MAXN : 0) + (GROUPED ? kRouteWarps * kGroupSpace<S> : 0)) +
                 w * RowFeed<S, Tl>::bytes(x.wide),
             full_s + w * 2);
  bool left = false;
  for (; t < T; t += step) {
    float l[V], c[V];
    // (by logits, NaN stay: they fail every comparison)
    if (!feed.template take<BY != kByLogit>(x, t, step, T, N, lane, l)) return;
    float m = 0.f, inv_z = 1.f;
    if constexpr (BY == kBySoftmax) {
      m = row_max<S>(l);
      const float z = row_softmax<S>(l, m, c);
      inv_z = z > 0.f ? rcp_fast(z) : 0.f;
    }
    if constexpr (SCORED) {
      float b[V];
      load_cells<S>(route_smem, q, b);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float s = BY == kBySoftmax ? fmaf(c[v], inv_z, b[v]) : sigmoid_fast(l[v]) + b[v];
        c[v] = masked_logit(l[v]) ? -INFINITY : s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = l[i];
    }
    // the sum of the row's exp(l - m) in 64 bits
    auto row_z64 = [&]() {
      double z = 0.0;
#pragma unroll 1
      for (int e = q; e < N; e += LPR) {
        const float v = x.at(t, e);
        if (!masked_logit(v)) z += score_64(v, m, 1.0, true);
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) z += __shfl_xor_sync(FULL_MASK, z, o);
      return z;
    };
    // The kept groups (bit g) by 64-bit values, for rows whose groups are too
    // near each other (about 1 in 10^4); by all lanes, needs room for the
    // values (fits_64).
    auto groups_64 = [&]() -> unsigned long long {
      if constexpr (!GROUPED || !SCORED) return 0ull;
      constexpr int GH = BFMOE_MAX_GROUPS / LPR;
      const double z64 = softmax ? row_z64() : 1.0;
      double* gd = reinterpret_cast<double*>(gs);
      __syncwarp();
#pragma unroll 1
      for (int cc = 0; cc < C; ++cc) {
        double a = -INFINITY, b = -INFINITY;
#pragma unroll 1
        for (int i = 0; i < CE; ++i) {
          const int e = (cc * LPR + q) * CE + i;
          double v = -INFINITY;
          if (e < N) {
            const float le = x.at(t, e);
            if (!masked_logit(le)) v = score_64(le, m, z64, softmax) + static_cast<double>(route_smem[slot_of<S>(e)]);
            if (!cells) gd[e] = v;
          }
          b = fmax(b, fmin(a, v));
          a = fmax(a, v);
        }
        if (cells) {
          gd[2 * (cc * LPR + q)] = a;
          gd[2 * (cc * LPR + q) + 1] = b;
        }
      }
      __syncwarp();
      // lane q: groups q, q + LPR, ...
      double gv64[GH];
      int r64[GH];
#pragma unroll
      for (int h = 0; h < GH; ++h) {
        double a = -INFINITY, b = -INFINITY;
        const int g = q + h * LPR;
#pragma unroll 1
        for (int it = 0; g < cfg.n_groups && it < items; ++it) {
          const double oa = cells ? gd[2 * (g * items + it)] : gd[g * items + it];
          const double ob = cells ? gd[2 * (g * items + it) + 1] : -INFINITY;
          b = fmax(fmin(a, oa), fmax(b, ob));
          a = fmax(a, oa);
        }
        gv64[h] = top2 && b > -INFINITY ? a + b : a;
        r64[h] = 0;
      }
#pragma unroll
      for (int h = 0; h < GH; ++h)
#pragma unroll 1
        for (int o = 0; o < min(cfg.n_groups - h * LPR, LPR); ++o) {
          const double v = __shfl_sync(FULL_MASK, gv64[h], o, LPR);
#pragma unroll
          for (int u = 0; u < GH; ++u)
            r64[u] += v > gv64[u] || (v == gv64[u] && o + h * LPR < q + u * LPR);
        }
      unsigned long long kept64 = 0ull;  // bit g
#pragma unroll
      for (int h = 0; h < GH; ++h)
        kept64 |= static_cast<unsigned long long>(
                      seg_bits<LPR>(q + h * LPR < cfg.n_groups && r64[h] < cfg.top_groups, lane))
                  << (h * LPR);
      return kept64;
    };
    // groups: the two best of each cell (or every value) go to shared memory,
    // lpg lanes take a group
    bool clear = true;
    unsigned allowed = V == 32 ? 0xffffffffu : (1u << V) - 1u;
    unsigned long long kept = ~0ull;  // bit g << lsh
    if (GROUPED && by_lanes) {
      // a group is 1 << lsh neighbouring lanes, each of one cell
      float a = -INFINITY, b = -INFINITY;
#pragma unroll
      for (int i = 0; i < CE; ++i) {
        b = fmaxf(b, fminf(a, c[i]));
        a = fmaxf(a, c[i]);
      }
#pragma unroll 1
      for (int o = 1; o < lpg; o <<= 1) {
        const float oa = __shfl_xor_sync(FULL_MASK, a, o), ob = __shfl_xor_sync(FULL_MASK, b, o);
        b = fmaxf(fminf(a, oa), fmaxf(b, ob));
        a = fmaxf(a, oa);
      }
      const float gv = group_worth(a, b, top2);
      int rank = 0;
#pragma unroll 1
      for (int o0 = 0; o0 < cfg.n_groups; o0 += lpg) {  // the lanes of a group share the comparisons
        const int o = o0 + (q & (lpg - 1));
        const float v = __shfl_sync(FULL_MASK, gv, (o << lsh) & 31);
        rank += o < cfg.n_groups && (v > gv || (v == gv && o < gq));
      }
#pragma unroll 1
      for (int o = 1; o < lpg; o <<= 1) rank += __shfl_xor_sync(FULL_MASK, rank, o);
      const bool real = gq < cfg.n_groups;
      bool in = real && rank < cfg.top_groups;
      if constexpr (SCORED) {
        const float eps = group_eps(eps_s, softmax, a, b);
        const float worst = -seg_max<LPR>(in ? -at_least(gv, eps) : -INFINITY);
        const float best = seg_max<LPR>(real && !in ? at_most(gv, eps) : -INFINITY);
        clear = !(best > -INFINITY) || worst > best;
        if (!clear) in = (groups_64() >> gq) & 1ull;
        clear = true;
        if (!bias) {
#pragma unroll
          for (int i = 0; i < V; ++i) c[i] = l[i];
        }
      }
      if (!in) {
        allowed = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = -INFINITY;
      }
    } else if constexpr (GROUPED) {
      if (cells) {
#pragma unroll
        for (int cc = 0; cc < C; ++cc) {
          float a = -INFINITY, b = -INFINITY;
#pragma unroll
          for (int i = 0; i < CE; ++i) {
            const float v = c[cc * CE + i];
            b = fmaxf(b, fminf(a, v));
            a = fmaxf(a, v);
          }
          *reinterpret_cast<float2*>(gs + 2 * (cc * LPR + q)) = make_float2(a, b);
        }
      } else {
#pragma unroll
        for (int cc = 0; cc < C; ++cc)
#pragma unroll
          for (int i = 0; i < CE; ++i) gs[(cc * LPR + q) * CE + i] = c[cc * CE + i];
      }
      __syncwarp();
      constexpr int GH = BFMOE_MAX_GROUPS / LPR;  // groups of a lane, at most
      const int hs = lsh == 0 ? (cfg.n_groups + LPR - 1) / LPR : 1;
      float gv[GH], eps[GH];
      int rank[GH];
#pragma unroll
      for (int h = 0; h < GH; ++h) {
        gv[h] = -INFINITY;
        rank[h] = 0;
        if (h >= hs) continue;
        const int g = gq + h * LPR;
        float a = -INFINITY, b = -INFINITY;
        if (g < cfg.n_groups) {
          for (int it = q & (lpg - 1); it < items; it += lpg) {
            float2 o = make_float2(-INFINITY, -INFINITY);
            if (cells) o = *reinterpret_cast<const float2*>(gs + 2 * (g * items + it));
            else o.x = gs[g * items + it];
            b = fmaxf(fminf(a, o.x), fmaxf(b, o.y));
            a = fmaxf(a, o.x);
          }
        }
        for (int o = 1; o < lpg; o <<= 1) {
          const float oa = __shfl_xor_sync(FULL_MASK, a, o), ob = __shfl_xor_sync(FULL_MASK, b, o);
          b = fmaxf(fminf(a, oa), fmaxf(b, ob));
          a = fmaxf(a, oa);
        }
        gv[h] = group_worth(a, b, top2);
        eps[h] = group_eps(eps_s, softmax, a, b);
      }
#pragma unroll
      for (int h = 0; h < GH; ++h) {
        if (h >= hs) continue;
        // the lanes of a group share the comparisons
        const int n = min(cfg.n_groups - h * LPR, LPR >> lsh);
        for (int o0 = 0; o0 < n; o0 += lpg) {
          const int o = o0 + (q & (lpg - 1));
          const float v = __shfl_sync(FULL_MASK, gv[h], min(o, n - 1) << lsh, LPR);
#pragma unroll
          for (int u = 0; u < GH; ++u)
            rank[u] += o < n && (v > gv[u] || (v == gv[u] && o + h * LPR < gq + u * LPR));
        }
      }
      for (int o = 1; o < lpg; o <<= 1) rank[0] += __shfl_xor_sync(FULL_MASK, rank[0], o);
      float worst = INFINITY, best = -INFINITY;  // of the kept, of the others
      kept = 0ull;
#pragma unroll
      for (int h = 0; h < GH; ++h) {
        if (h >= hs) continue;
        const bool real = gq + h * LPR < cfg.n_groups && (q & (lpg - 1)) == 0;
        const bool in = real && rank[h] < cfg.top_groups;
        if (in) worst = fminf(worst, at_least(gv[h], eps[h]));
        else if (real) best = fmaxf(best, at_most(gv[h], eps[h]));
        kept |= static_cast<unsigned long long>(seg_bits<LPR>(in, lane)) << (h * LPR);
      }
      if constexpr (SCORED) {
        worst = -seg_max<LPR>(-worst);
        best = seg_max<LPR>(best);
        clear = !(best > -INFINITY) || worst > best;
        if (!clear && fits_64) {
          const unsigned long long kept64 = groups_64();
          kept = 0ull;
          for (int g = 0; g < cfg.n_groups; ++g) kept |= ((kept64 >> g) & 1ull) << (g << lsh);
          clear = true;
        }
        if (!bias) {
#pragma unroll
          for (int i = 0; i < V; ++i) c[i] = l[i];
        }
      }
    }
    // what is no candidate: the other groups, and nothing behind the row's end
    if ((GROUPED && !by_lanes) || N < S::MAXN) {
      const unsigned before = allowed;
      allowed = 0u;
#pragma unroll
      for (int cc = 0; cc < C; ++cc) {
        const int e0 = (cc * LPR + q) * CE;
        unsigned in = e0 + CE <= N ? (1u << CE) - 1u : (e0 < N ? (1u << (N - e0)) - 1u : 0u);
        if constexpr (GROUPED) {
          if (by_lanes) {
            in &= before;
          } else if (cells) {
            if (!((kept >> (g0[cc] << lsh)) & 1ull)) in = 0u;
          } else if (in) {
            int g = g0[cc], r = e0 - g * per;
            bool on = (kept >> (g << lsh)) & 1ull;
#pragma unroll
            for (int i = 0; i < CE; ++i) {
              if (r == per) {
                r = 0;
                ++g;
                on = e0 + i < N && ((kept >> (g << lsh)) & 1ull);
              }
              ++r;
              if (!on) in &= ~(1u << i);
            }
          }
        }
        allowed |= in << (cc * CE);
      }
    }
    if (GROUPED && !by_lanes) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!((allowed >> i) & 1u)) c[i] = -INFINITY;
    }
    float h = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) h = fmaxf(h, c[i]);
    // threshold
    const uint32_t first = ordered(h);
    uint32_t key = first, last = 0u;
#pragma unroll 1
    for (int have = 0; have <= k;) {
      last = __reduce_max_sync(FULL_MASK, key);
      have += __popc(__ballot_sync(FULL_MASK, key == last));
      if (key == last) key = 0u;
    }
    float least = from_ordered(last);
    if (least == -INFINITY && N > 32) {
      // what is left of the row lies in few lanes (groups, masks): the same
      // over all values
      float top = INFINITY;
#pragma unroll 1
      for (int have = 0; have <= k;) {
        float v = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (c[i] < top || have == 0) v = fmaxf(v, c[i]);
        top = seg_max<LPR>(v);
        if (top == -INFINITY) break;
        int equal = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) equal += c[i] == top;
        have += __reduce_add_sync(FULL_MASK, equal);
      }
      least = top;
    }
    if constexpr (SCORED) {
      if (bias && least < INFINITY) least -= 2.f * value_eps(eps_s, softmax, 1.f, least);
    }
    // who reaches it: bit V - 1 - i for value i (the sign of the difference to
    // the next lower number: 0 and -0 are equal, and so is who is it)
    unsigned want = 0u;
    if (fabsf(least) < INFINITY) {
      least = from_ordered(ordered(least) - 1u);
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 d = __fadd2_rn(pair(c, i), make_float2(-least, -least));
        want = __funnelshift_l(__float_as_uint(d.x), want, 1);
        want = __funnelshift_l(__float_as_uint(d.y), want, 1);
      }
      want = ~want;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) want = want << 1 | (least < 0.f || c[i] == least);
    }
    want &= __brev(allowed) >> (32 - V);
    // candidates into lanes
    int n = 0;
    for (;;) {
      const unsigned b = __ballot_sync(FULL_MASK, want != 0u);
      if (!b) break;
      const int at = n + __popc(b & ((1u << lane) - 1u));
      if (want) {
        const int i = V - __ffs(want);
        if (at < 32) cand[at].e = ((i / CE) * LPR + lane) * CE + i % CE;
        want &= want - 1u;
      }
      n += __popc(b);
      if (n > 32) break;
    }
    __syncwarp();
    clear = clear && n <= 32;
    n = min(n, 32);
    if constexpr (BY == kByLogit) {
      if (softmax && !cfg.renorm) {
        if constexpr (GROUPED) m = row_max<S>(l);
        else m = from_ordered(__reduce_max_sync(FULL_MASK, first));
        float z = row_softmax<S>(l, m, c);
        if (z != z) {  // NaN among the logits
#pragma unroll
          for (int i = 0; i < V; ++i) l[i] = fmaxf(l[i], -INFINITY);
          z = row_softmax<S>(l, m, c);
        }
        inv_z = z > 0.f ? rcp_fast(z) : 0.f;
      }
    }
    int e = 0x7fffffff;
    float le = -INFINITY, sc = 0.f, val = -INFINITY, eps = 0.f;
    if (lane < n) {
      e = cand[lane].e;
      le = feed.at(x, t, e);
      if (masked_logit(le)) le = -INFINITY;  // NaN
      if (bias || !cfg.renorm) sc = softmax ? (le > -INFINITY ? unit_softmax(le, m) * inv_z : 0.f) : sigmoid_fast(le);
      val = le;
      if constexpr (SCORED) {
        if (bias && le > -INFINITY) {
          val = sc + route_smem[slot_of<S>(e)];
          eps = value_eps(eps_s, softmax, sc, val);
        }
      }
      cand[lane] = Candidate{val, e, eps, 0};
    }
    __syncwarp();
    int rank = lane < n ? 0 : 32, near = 0;
#pragma unroll 4
    for (int o = 0; o < n; ++o) {
      const Candidate a = cand[o];
      rank += a.value > val || (a.value == val && a.e < e);
      if constexpr (SCORED) near += !(fabsf(a.value - val) > a.eps + eps);
    }
    if constexpr (SCORED) {
      // (a value is near itself; masked ones, -inf, are near each other: so is
      // what infinities make)
      if (bias && __any_sync(FULL_MASK, lane < n && near > 1 && val > -INFINITY)) {
        const double z64 = softmax ? row_z64() : 1.0;
        double v64 = -INFINITY;
        if (val > -INFINITY) v64 = score_64(le, m, z64, softmax) + static_cast<double>(route_smem[slot_of<S>(e)]);
        rank = lane < n ? 0 : 32;
        for (int o = 0; o < n; ++o) {
          const double ov = __shfl_sync(FULL_MASK, v64, o);
          const int oe = __shfl_sync(FULL_MASK, e, o);
          rank += ov > v64 || (ov == v64 && oe < e);
        }
      }
    }
    const bool mine = rank < k && val > -INFINITY;
    float u = 0.f;
    if (cfg.renorm) {
      const float top = seg_max<LPR>(mine ? le : -INFINITY);
      if (mine) u = softmax ? unit_softmax(le, top) : unit_sigmoid(le, fminf(top, 0.f));
      const float sum = seg_sum<LPR>(u);
      u = sum > 0.f ? u * rcp_fast(sum) : 0.f;
    } else if (mine) {
      u = sc;
    }
    if (clear) {
      if (rank < k) {
        idx[static_cast<long long>(t) * k + rank] = e;
        gates[static_cast<long long>(t) * k + rank] = u * cfg.scale;
      }
    } else {
      if (lane == 0) idx[static_cast<long long>(t) * k] = -1;
      left = true;
    }
    __syncwarp();  // the candidates and group values are read before the next row's are written
  }
  if (!left) return;
  // the rows left over (marked by the warp itself above)
  for (t = blockIdx.x * kRouteWarps + w; t < T; t += step) {
    if (__shfl_sync(FULL_MASK, lane == 0 ? idx[static_cast<long long>(t) * k] : 0, 0) >= 0) continue;
    int e;
    float g;
    route_row_64(x, t, N, k, cfg, bias, reinterpret_cast<int*>(cand), lane, e, g);
    if (lane < k) {
      idx[static_cast<long long>(t) * k + lane] = e;
      gates[static_cast<long long>(t) * k + lane] = g;
    }
  }
}

// Rows of more experts than registers hold: a warp a row, several passes over
// it (it stays in the caches).
template <typename Tl>
__global__ __launch_bounds__(kRouteWarps * 32) void route_long_kernel(const Logits<Tl> x, int T, int N, int k,
                                                                      const RouteCfg cfg,
                                                                      const float* __restrict__ bias,
                                                                      int32_t* __restrict__ idx,
                                                                      float* __restrict__ gates) {
  __shared__ int win_s[kRouteWarps][kRouteWindow];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  for (int t = blockIdx.x * kRouteWarps + w; t < T; t += gridDim.x * kRouteWarps) {
    int e;
    float g;
    route_row_64(x, t, N, k, cfg, bias, win_s[w], lane, e, g);
    if (lane < k) {
      idx[static_cast<long long>(t) * k + lane] = e;
      gates[static_cast<long long>(t) * k + lane] = g;
    }
  }
}

}  // namespace bfmoe
