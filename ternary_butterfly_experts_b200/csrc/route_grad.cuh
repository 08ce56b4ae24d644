// Gradient of the routing (route.cuh) and the losses that keep the experts in
// use.
//
// Gates, the choice held: with r_j the gates over the scale,
//   renormalised softmax  dl_j = scale r_j (dg_j - sum r dg)
//   renormalised sigmoid  the same times (1 - s_j)
//   plain softmax         dl_e = p_e ([e chosen] scale dg_e - sum_j scale p_j dg_j)
//   plain sigmoid         dl_j = scale dg_j s_j (1 - s_j)
// Losses over the R rows that have an expert left, p the scores over their
// sum, f_e = load_e / (k R) the share of slots that went to expert e (a count:
// no gradient):
//   balance  N sum_e f_e mean_t p_te    dl_e = N / R p_e (f_e - sum f p)  [sigmoid: times 1 - s_e]
//   z        mean_t lse_t^2             dl_e = 2 / R lse softmax_e
#pragma once
#include "route.cuh"

namespace bfmoe {

constexpr int kGradWarps = 8;
template <class S>
constexpr int kGradRowBlocks = S::V <= 8 ? 4 : (S::V <= 16 ? 3 : 2);  // of an SM
template <class S>
constexpr int kBalanceRowBlocks = S::V <= 8 ? 4 : (S::V <= 16 ? 3 : 2);

// lse of a row from its largest logit and sum of exp(l - m).
__device__ __forceinline__ float row_lse(float m, float z) { return m + __logf(z); }

// e^-|l| and 1 / (1 + e^-|l|): sigmoid(l) and sigmoid(-l) without cancellation.
struct TwoSided {
  float s, t;  // sigmoid(l), sigmoid(-l)
  __device__ __forceinline__ explicit TwoSided(float l) {
    const float e = exp_fast(-fabsf(l)), r = rcp_fast(1.f + e);
    s = l > 0.f ? r : e * r;
    t = l > 0.f ? e * r : r;
  }
};
// The row's sigmoids up to a factor of the row (shares need no more) in u,
// sigmoid(-l) in t; masked logits give 0 and 1.  Where softmax terms x =
// exp(l - m) are at hand and the largest logit is moderate, sigmoid(l) is
// x / (x + exp(-m)): no second exponential.
__device__ __forceinline__ bool moderate(float m) { return !__any_sync(FULL_MASK, !(m >= -10.f && m <= 20.f)); }
// 1 / (x + c) for a row's x in [0, 1] and c in [e^-20, e^10], in r: four
// reciprocals from one (products of four stay within float32; the special
// function unit, 16 results a clock and SM, is what bounds the losses).
template <class S>
__device__ __forceinline__ void row_reciprocals(const float (&x)[S::V], float c, float (&r)[S::V]) {
#pragma unroll
  for (int i = 0; i < S::V; i += 4) {
    const float2 c2 = make_float2(c, c);
    const float2 a = __fadd2_rn(pair(x, i), c2), b = __fadd2_rn(pair(x, i + 2), c2);
    const float p = a.x * a.y, q = b.x * b.y, one = rcp_fast(p * q);
    const float rp = one * q, rq = one * p;
    r[i] = rp * a.y;
    r[i + 1] = rp * a.x;
    r[i + 2] = rq * b.y;
    r[i + 3] = rq * b.x;
  }
}
template <class S>
__device__ __forceinline__ void row_sigmoid(const float (&l)[S::V], float m, bool has_x, const float (&x)[S::V],
                                            float (&u)[S::V], float (&t)[S::V]) {
  if (has_x && moderate(m)) {
    const float c = exp_fast(-m);
    row_reciprocals<S>(x, c, t);
#pragma unroll
    for (int i = 0; i < S::V; i += 2) {
      const float2 r = pair(t, i), s = __fmul2_rn(pair(x, i), r), o = __fmul2_rn(make_float2(c, c), r);
      u[i] = s.x, u[i + 1] = s.y;
      t[i] = o.x, t[i + 1] = o.y;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < S::V; ++i) {
    const TwoSided v(l[i]);
    u[i] = v.s;
    t[i] = v.t;
  }
  if (m < 0.f && m > -INFINITY) {
#pragma unroll
    for (int i = 0; i < S::V; ++i) u[i] = masked_logit(l[i]) ? 0.f : exp_fast(l[i] - m) * t[i];
  }
}
// One pass over the logits: the sums of the losses' terms over this block's
// rows, in a fixed order: part [grid][N] of p_te, zpart [grid] of lse^2, and
// loads [grid][N + 1], the chosen slots of each expert and the rows.  A lane
// keeps the sums of its experts in registers.  131072 x 1024 float32, sigmoid
// scores: 107 us, 5.0 TB/s; bound by the special function unit (1.25 results a
// logit) and the instructions around it, at 16 warps an SM.
template <class S, typename Tl, bool SIGMOID>
__global__ __launch_bounds__(kGradWarps * 32, kBalanceRowBlocks<S>) void balance_rows_kernel(
    const Logits<Tl> x, int T, int N, int k, const int32_t* __restrict__ idx, float* __restrict__ part,
    double* __restrict__ zpart, int32_t* __restrict__ loads) {
  constexpr int LPR = S::LPR, V = S::V;
  extern __shared__ __align__(128) float grad_smem[];  // sums of a warp [kGradWarps][MAXN]; during the rows: their buffers
  __shared__ int hist[S::MAXN];
  __shared__ double zs[kGradWarps];
  __shared__ int rs[kGradWarps];
  __shared__ uint64_t full_s[kGradWarps * 2];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, q = lane & (LPR - 1);
  for (int e = threadIdx.x; e < S::MAXN; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.f;
  double z2 = 0.0;
  int rows = 0;
  const int step = gridDim.x * kGradWarps * S::ROWS;
  int t0 = (blockIdx.x * kGradWarps + w) * S::ROWS;
  RowFeed<S, Tl> feed;
  feed.start(x, t0, T, N, lane, reinterpret_cast<uint8_t*>(grad_smem) + w * RowFeed<S, Tl>::bytes(x.wide),
             full_s + w * 2);
  auto slot = [&](int t) { return q < k && t < T ? idx[static_cast<long long>(t) * k + q] : -1; };
  int e = slot(t0 + lane / LPR);
  for (; t0 < T; t0 += step) {
    const int t = t0 + lane / LPR;
    float l[V], u[V];
    if (!feed.take(x, t0, step, T, N, lane, l)) break;
    const int e_now = e;
    e = slot(t + step);
    float m = row_max<S>(l);
    // (a row past the end, anything, has no say in how the others are worked out)
    if (SIGMOID && t >= T) m = 0.f;
    const bool some = t < T && m > -INFINITY;
    const float z = row_softmax<S>(l, m, u);
    float inv;
    if constexpr (SIGMOID) {
      if (moderate(m)) {
        float r[V];
        row_reciprocals<S>(u, exp_fast(-m), r);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 s = __fmul2_rn(pair(u, i), pair(r, i));
          u[i] = s.x, u[i + 1] = s.y;
        }
      } else {
        float c[V];
        feed.again(x, min(t, T - 1), N, lane, l);
        row_sigmoid<S>(l, m, false, u, u, c);
      }
      inv = rcp_fast(seg_sum<LPR>(lane_sum(u)));
    } else {
      inv = rcp_fast(z);
    }
    if (some) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 s = __ffma2_rn(pair(u, i), make_float2(inv, inv), pair(sum, i));
        sum[i] = s.x, sum[i + 1] = s.y;
      }
      if (q < k) {
        if (e_now >= 0 && e_now < N) atomicAdd(hist + e_now, 1);
        else report_error(BFMOE_EDEVICE_BOUNDS, static_cast<unsigned>(t));
      }
      if (q == 0) {
        const double lse = static_cast<double>(row_lse(m, z));
        z2 += lse * lse;
        ++rows;
      }
    }
  }
  // lanes, then warps
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] += __shfl_xor_sync(FULL_MASK, sum[i], o);
    z2 += __shfl_xor_sync(FULL_MASK, z2, o);
    rows += __shfl_xor_sync(FULL_MASK, rows, o);
  }
  __syncthreads();  // the row buffers are read
  if (lane < LPR) {
#pragma unroll
    for (int c = 0; c < S::C; ++c)
#pragma unroll
      for (int h = 0; h < S::CE; h += 4)
        *reinterpret_cast<float4*>(grad_smem + w * S::MAXN + (c * LPR + q) * S::CE + h) =
            make_float4(sum[c * S::CE + h], sum[c * S::CE + h + 1], sum[c * S::CE + h + 2], sum[c * S::CE + h + 3]);
  }
  if (lane == 0) {
    zs[w] = z2;
    rs[w] = rows;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < N; i += blockDim.x) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kGradWarps; ++v) s += grad_smem[v * S::MAXN + i];
    part[static_cast<size_t>(blockIdx.x) * N + i] = s;
    loads[static_cast<size_t>(blockIdx.x) * (N + 1) + i] = hist[i];
  }
  if (threadIdx.x == 0) {
    double s = 0.0;
    int r = 0;
    for (int v = 0; v < kGradWarps; ++v) {
      s += zs[v];
      r += rs[v];
    }
    zpart[blockIdx.x] = s;
    loads[static_cast<size_t>(blockIdx.x) * (N + 1) + N] = r;
  }
}

// Sums of one row, by a warp, for rows of more experts than registers hold.
struct RowSums {
  float m, z, s;  // largest logit, sum of unit_softmax, sum of unit_sigmoid
};
template <typename Tl>
__device__ __forceinline__ RowSums row_sums(const Logits<Tl>& x, int t, int N, int lane, bool sigmoid) {
  RowSums r;
  float m = -INFINITY;
  for (int e = lane; e < N; e += 32) m = fmaxf(m, x.at(t, e));
  r.m = warp_max(m);
  const float low = fminf(r.m, 0.f);
  float z = 0.f, s = 0.f;
  for (int e = lane; e < N; e += 32) {
    const float l = x.at(t, e);
    if (masked_logit(l)) continue;
    z += unit_softmax(l, r.m);
    if (sigmoid) s += unit_sigmoid(l, low);
  }
  r.z = warp_sum(z);
  r.s = sigmoid ? warp_sum(s) : r.z;
  return r;
}

// balance_rows_kernel for such rows: a warp a row, the sums in shared memory.
template <typename Tl>
__global__ __launch_bounds__(kGradWarps * 32) void balance_long_kernel(const Logits<Tl> x, int T, int N, int k, int sig,
                                                                       const int32_t* __restrict__ idx,
                                                                       float* __restrict__ part,
                                                                       double* __restrict__ zpart,
                                                                       int32_t* __restrict__ loads) {
  extern __shared__ __align__(128) float grad_smem[];  // [kGradWarps][N], then the counts [N]
  __shared__ double zs[kGradWarps];
  __shared__ int rs[kGradWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int* hist = reinterpret_cast<int*>(grad_smem + static_cast<size_t>(kGradWarps) * N);
  float* mine = grad_smem + static_cast<size_t>(w) * N;
  for (int e = lane; e < N; e += 32) mine[e] = 0.f;
  for (int e = threadIdx.x; e < N; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  double z2 = 0.0;
  int rows = 0;
  for (int t = blockIdx.x * kGradWarps + w; t < T; t += gridDim.x * kGradWarps) {
    const RowSums r = row_sums(x, t, N, lane, sig != 0);
    if (!(r.m > -INFINITY)) continue;
    const float low = fminf(r.m, 0.f), inv = 1.f / r.s;
    for (int e = lane; e < N; e += 32) {
      const float l = x.at(t, e);
      if (!masked_logit(l)) mine[e] += (sig ? unit_sigmoid(l, low) : unit_softmax(l, r.m)) * inv;
    }
    const double lse = static_cast<double>(row_lse(r.m, r.z));
    z2 += lse * lse;
    ++rows;
    if (lane < k) {
      const int e = idx[static_cast<long long>(t) * k + lane];
      if (e >= 0 && e < N) atomicAdd(hist + e, 1);
      else report_error(BFMOE_EDEVICE_BOUNDS, static_cast<unsigned>(t));
    }
  }
  if (lane == 0) {
    zs[w] = z2;
    rs[w] = rows;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < N; e += blockDim.x) {
    float s = 0.f;
    for (int v = 0; v < kGradWarps; ++v) s += grad_smem[static_cast<size_t>(v) * N + e];
    part[static_cast<size_t>(blockIdx.x) * N + e] = s;
    loads[static_cast<size_t>(blockIdx.x) * (N + 1) + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    double s = 0.0;
    int r = 0;
    for (int v = 0; v < kGradWarps; ++v) {
      s += zs[v];
      r += rs[v];
    }
    zpart[blockIdx.x] = s;
    loads[static_cast<size_t>(blockIdx.x) * (N + 1) + N] = r;
  }
}

// The blocks' sums added up, by one cluster; each of its blocks takes a share
// of the experts, its threads slices of the rows of part and loads.
constexpr int kFinishBlocks = 8;
constexpr int kFinishThreads = 1024;
__global__ __cluster_dims__(kFinishBlocks, 1, 1) __launch_bounds__(kFinishThreads) void balance_finish_kernel(
    const float* __restrict__ part, const double* __restrict__ zpart, const int32_t* __restrict__ loads, int blocks,
    int N, int k, int32_t* __restrict__ load, float* __restrict__ loss) {
  __shared__ double ps[kFinishThreads];
  __shared__ int ls[kFinishThreads];
  __shared__ double share[kFinishBlocks];  // of block 0: each block's sum of load P
  const int rank = blockIdx.x, tid = threadIdx.x;
  const int per = (N + kFinishBlocks - 1) / kFinishBlocks;  // <= 512
  int width = 1;
  while (width < per) width <<= 1;
  const int slices = kFinishThreads / width, e = rank * per + (tid & (width - 1)), slice = tid / width;
  const bool real = (tid & (width - 1)) < per && e < N;
  // (waited for before the store into block 0's memory: block 0 runs by then)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  pdl_trigger();
  double p = 0.0;
  int c = 0;
  if (real)
    for (int b = slice; b < blocks; b += slices) {
      p += static_cast<double>(part[static_cast<size_t>(b) * N + e]);
      c += loads[static_cast<size_t>(b) * (N + 1) + e];
    }
  ps[tid] = p;
  ls[tid] = c;
  __syncthreads();
  for (int s = kFinishThreads / 2; s >= width; s >>= 1) {
    if (tid < s) {
      ps[tid] += ps[tid + s];
      ls[tid] += ls[tid + s];
    }
    __syncthreads();
  }
  double mine = 0.0;
  if (tid < width && real) {
    load[e] = ls[tid];
    mine = ps[tid] * static_cast<double>(ls[tid]);
  }
  __syncthreads();
  ps[tid] = mine;
  __syncthreads();
  for (int s = kFinishThreads / 2; s > 0; s >>= 1) {
    if (tid < s) ps[tid] += ps[tid + s];
    __syncthreads();
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (tid == 0) {
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"(smem_u32(share + rank)));
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(there), "d"(ps[0]) : "memory");
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0) {
    // rows and z, a warp each
    double z = 0.0;
    int r = 0;
    if (tid < 32)
      for (int b = tid; b < blocks; b += 32) {
        z += zpart[b];
        r += loads[static_cast<size_t>(b) * (N + 1) + N];
      }
    if (tid < 32) {
      z = warp_sum(z);
      r = __reduce_add_sync(FULL_MASK, r);
      if (tid == 0) {
        double b = 0.0;
        for (int q = 0; q < kFinishBlocks; ++q) b += share[q];
        const double R = static_cast<double>(r);
        load[N] = r;
        loss[0] = r > 0 ? static_cast<float>(b * N / (static_cast<double>(k) * R * R)) : 0.f;
        loss[1] = r > 0 ? static_cast<float>(z / R) : 0.f;
      }
    }
  }
}

// CE consecutive float32 values to an aligned cell.  (Eight in one store: as
// two, each wrote half of every 32-byte sector that it touched.)
template <int CE>
__device__ __forceinline__ void store_cell(float* p, const float* v) {
  if constexpr (CE == 8) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
}
template <int CE>
__device__ __forceinline__ void store_cell(__nv_bfloat16* p, const float* v) {
  uint32_t b[CE / 2];
#pragma unroll
  for (int h = 0; h < CE / 2; ++h) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * h], v[2 * h + 1]);
    b[h] = *reinterpret_cast<const uint32_t*>(&x);
  }
  if constexpr (CE == 8) *reinterpret_cast<uint4*>(p) = make_uint4(b[0], b[1], b[2], b[3]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(b[0], b[1]);
}

struct RouteGrad {
  const int32_t* idx;
  const float* bias;     // balance bias, or NULL: only where it masks
  const float* dgates;   // or NULL
  const int32_t* load;   // or NULL
  const float* dloss;
  void* out;
  long long ld_out;
  int wide_out;
};

// Factors of the losses: balance times N / R and 1 / (k R), z times 2 / R.
struct LossFactors {
  float cb, cz;
  __device__ __forceinline__ LossFactors(const RouteGrad& g, int N, int k) {
    cb = cz = 0.f;
    if (g.load) {
      const float R = static_cast<float>(g.load[N]);
      if (R > 0.f) {
        cb = g.dloss[0] * static_cast<float>(N) / R / (static_cast<float>(k) * R);
        cz = 2.f * g.dloss[1] / R;
        if (!(fabsf(cb) < INFINITY)) {
          // NaN for every expert that has a score: it comes through the z loss's
          // factor, which masked experts do not meet
          cz = cb - cb;
          cb = 0.f;
        }
      }
    }
  }
};

// The gradient of row t by one warp, in several passes over the row.
template <typename Tl>
__device__ __noinline__ void route_backward_row(const Logits<Tl>& x, int t, int N, int k, const RouteCfg& cfg,
                                                const RouteGrad& g, LossFactors f, int lane) {
  const bool sig = cfg.score == BFMOE_SCORE_SIGMOID;
  const bool dense = g.dgates && !sig && !cfg.renorm;
  RowSums r{-INFINITY, 0.f, 0.f};
  if (g.load || dense) r = row_sums(x, t, N, lane, sig);
  const float low = fminf(r.m, 0.f);
  const float inv_z = r.z > 0.f ? 1.f / r.z : 0.f, inv_s = r.s > 0.f ? 1.f / r.s : 0.f;
  int e = -1;
  float d = 0.f, dot = 0.f;
  if (g.dgates) {
    float l = -INFINITY, dg = 0.f;
    if (lane < k) {
      e = g.idx[static_cast<long long>(t) * k + lane];
      if (e < 0 || e >= N) {
        report_error(BFMOE_EDEVICE_BOUNDS, static_cast<unsigned>(t));
        e = -1;
      } else {
        l = x.at(t, e);
        dg = g.dgates[static_cast<long long>(t) * k + lane] * cfg.scale;
      }
    }
    const bool live = e >= 0 && !masked_logit(l) && !(g.bias && masked_logit(g.bias[e]));
    if (!live) dg = 0.f;
    if (dense) {
      d = live ? unit_softmax(l, r.m) * inv_z * dg : 0.f;
      dot = warp_sum(d);
    } else if (cfg.renorm) {
      const float m = warp_max(live ? l : -INFINITY);
      const float u = !live ? 0.f : (sig ? unit_sigmoid(l, fminf(m, 0.f)) : unit_softmax(l, m));
      const float s = warp_sum(u);
      const float q = s > 0.f ? u / s : 0.f;
      const float mean = warp_sum(q * dg);
      d = q != 0.f ? q * (dg - mean) : 0.f;
    } else {
      d = live ? dg * sigmoid_fast(l) : 0.f;
    }
    if (sig) d = live ? d * sigmoid_fast(-l) : 0.f;
  }
  float pa = 0.f;
  if (f.cb != 0.f) {
    for (int q = lane; q < N; q += 32) {
      const float l = x.at(t, q);
      if (masked_logit(l)) continue;
      pa += (sig ? unit_sigmoid(l, low) : unit_softmax(l, r.m)) * inv_s * (f.cb * static_cast<float>(g.load[q]));
    }
    pa = warp_sum(pa);
  }
  const float lse = f.cz != 0.f ? f.cz * row_lse(r.m, r.z) : 0.f;
  __syncwarp();
  for (int q0 = 0; q0 < N; q0 += 32) {
    const int q = q0 + lane;
    float o = 0.f;
    if (q < N) {
      const float l = x.at(t, q);
      if (!masked_logit(l)) {
        const float p = dense || f.cb != 0.f || f.cz != 0.f ? unit_softmax(l, r.m) * inv_z : 0.f;
        // (where p is 0 the row's sums take no part, finite or not)
        if (dense && p != 0.f) o -= p * dot;
        if (f.cb != 0.f) {
          float ps = sig ? unit_sigmoid(l, low) * inv_s : p;
          if (sig) ps *= sigmoid_fast(-l);
          if (ps != 0.f) o += ps * (f.cb * static_cast<float>(g.load[q]) - pa);
        }
        if (p != 0.f) o += lse * p;
      }
    }
    for (int j = 0; j < k; ++j) {
      const int ej = __shfl_sync(FULL_MASK, e, j);
      const float dj = __shfl_sync(FULL_MASK, d, j);
      if (ej == q) o += dj;
    }
    if (q < N) {
      const long long at = static_cast<long long>(t) * g.ld_out + q;
      static_cast<Tl*>(g.out)[at] = from_f32<Tl>(o);
    }
  }
  __syncwarp();
}

// A row in registers: the gradient of every logit is p_e (a_e + K) from the
// losses and the plain softmax's gates (a_e = cb load_e, K the row's sums), and
// each chosen expert has its own term, which reaches its lane through shared
// memory.  Where only chosen experts have one (ROW false), the row is not read.
// 65536 x 256 float32, both losses and plain softmax gates: 32 us, 4.2 TB/s;
// bound by the latency of a row's sums and shared-memory passes (6 warps a
// scheduler), not by memory.
template <class S, typename Tl, bool SIGMOID, bool ROW>
__global__ __launch_bounds__(kGradWarps * 32, ROW ? kGradRowBlocks<S> : 4) void route_backward_kernel(
    const __grid_constant__ Logits<Tl> x, int T, int N, int k, const __grid_constant__ RouteCfg cfg,
    const __grid_constant__ RouteGrad g) {
  constexpr int LPR = S::LPR, V = S::V;
  extern __shared__ __align__(128) float grad_smem[];  // a [MAXN], the rows' chosen terms [warps * ROWS][MAXN], buffers
  __shared__ uint64_t full_s[kGradWarps * 2];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, q = lane & (LPR - 1);
  float* mine = grad_smem + S::MAXN + (w * S::ROWS + lane / LPR) * S::MAXN;
#pragma unroll
  for (int i = 0; i < V; ++i) mine[i * LPR + q] = 0.f;
  pdl_wait();
  pdl_trigger();
  const LossFactors f(g, N, k);
  for (int e = threadIdx.x; e < S::MAXN; e += blockDim.x)
    grad_smem[slot_of<S>(e)] = e < N && f.cb != 0.f ? f.cb * static_cast<float>(g.load[e]) : 0.f;
  __syncthreads();
  const bool dense = g.dgates && !SIGMOID && !cfg.renorm;  // every logit moves every gate
  const int step = gridDim.x * kGradWarps * S::ROWS;
  int t0 = (blockIdx.x * kGradWarps + w) * S::ROWS;
  RowFeed<S, Tl> feed;
  if constexpr (ROW)
    feed.start(x, t0, T, N, lane,
               reinterpret_cast<uint8_t*>(grad_smem + S::MAXN * (1 + kGradWarps * S::ROWS)) +
                   w * RowFeed<S, Tl>::bytes(x.wide),
               full_s + w * 2);
  // lane q < k holds slot q of its row.  Loads run ahead: a row's experts and
  // gate gradients by two rows, and, where the row itself is not read, the
  // logits of its experts by one.  (Nothing is computed from what was just
  // loaded: that would wait for it.)
  struct Slot {
    int e;
    float dg, l;
  } now{-1, 0.f, -INFINITY}, next{-1, 0.f, -INFINITY}, after{-1, 0.f, -INFINITY};
  auto ask = [&](Slot& s, int t) {
    s.e = -1;
    if (g.dgates && q < k && t < T) {
      s.e = g.idx[static_cast<long long>(t) * k + q];
      s.dg = g.dgates[static_cast<long long>(t) * k + q];
    }
  };
  auto ask_logit = [&](Slot& s, int t) {
    s.l = -INFINITY;
    if (!ROW && s.e >= 0 && s.e < N) s.l = x.at(t, s.e);
  };
  ask(next, t0 + lane / LPR);
  ask(after, t0 + step + lane / LPR);
  ask_logit(next, t0 + lane / LPR);
  for (; t0 < T; t0 += step) {
    const int t = min(t0 + lane / LPR, T - 1);
    const bool has = t0 + lane / LPR < T;
    float l[ROW ? V : 1], u[ROW ? V : 1], tt[ROW && SIGMOID ? V : 1];
    if constexpr (ROW) {
      if (!feed.take(x, t0, step, T, N, lane, l)) return;
    }
    now = next;
    next = after;
    ask_logit(next, t0 + step + lane / LPR);
    ask(after, t0 + 2 * step + lane / LPR);
    int e = now.e;
    // the chosen
    float le = -INFINITY;
    bool live = false;
    if (g.dgates) {
      if (q < k && has && (e < 0 || e >= N)) {
        report_error(BFMOE_EDEVICE_BOUNDS, static_cast<unsigned>(t));
        e = -1;
      }
      if (e >= 0) {
        if constexpr (ROW) le = feed.at(x, t, e);
        else le = now.l;
      }
      live = e >= 0 && !masked_logit(le) && !(g.bias && masked_logit(g.bias[e]));
    }
    const float dg = live ? now.dg * cfg.scale : 0.f;
    float m = 0.f, inv = 0.f, pa = 0.f, lse = 0.f;
    if constexpr (ROW) {
      m = row_max<S>(l);
      float s = 0.f;
      if constexpr (SIGMOID) {
        if (!has) m = 0.f;  // (past the end: no say in how the warp's other rows are worked out)
        if (f.cz != 0.f) {  // softmax_e lse cz is added at the end
          const float z = row_softmax<S>(l, m, u);
          lse = m > -INFINITY ? row_lse(m, z) * f.cz * rcp_fast(z) : 0.f;
        }
        row_sigmoid<S>(l, m, f.cz != 0.f, u, u, tt);
        s = seg_sum<LPR>(lane_sum(u));
      } else {
        s = row_softmax<S>(l, m, u);
        // (without a z loss not even of a row with +inf logits: inf times 0)
        lse = f.cz != 0.f && m > -INFINITY ? row_lse(m, s) * f.cz : 0.f;
      }
      inv = s > 0.f ? rcp_fast(s) : 0.f;
      if (f.cb != 0.f) {
        float b = 0.f;
#pragma unroll
        for (int c = 0; c < S::C; ++c) {
          float a[S::CE];
          load_cell_of<S>(grad_smem, q, c, a);
#pragma unroll
          for (int i = 0; i < S::CE; ++i) b = fmaf(u[c * S::CE + i], a[i], b);
        }
        pa = seg_sum<LPR>(b) * inv;
      }
    }
    float d = 0.f, dot = 0.f;
    if (g.dgates) {
      if (dense) {
        d = live ? unit_softmax(le, m) * inv * dg : 0.f;
        dot = seg_sum<LPR>(d);
      } else if (cfg.renorm) {
        const float top = seg_max<LPR>(live ? le : -INFINITY);
        const float v = !live ? 0.f : (SIGMOID ? unit_sigmoid(le, fminf(top, 0.f)) : unit_softmax(le, top));
        const float s = seg_sum<LPR>(v);
        const float r = s > 0.f ? v * rcp_fast(s) : 0.f;
        const float mean = seg_sum<LPR>(r * dg);
        d = r != 0.f ? r * (dg - mean) : 0.f;  // (a masked one has no part in a NaN either)
      } else {
        d = live ? dg * sigmoid_fast(le) : 0.f;
      }
      if (SIGMOID) d = live ? d * sigmoid_fast(-le) : 0.f;
      // the terms of one expert chosen twice add up in slot order
      float all = 0.f;
      for (int o = 0; o < k; ++o) {
        const int eo = __shfl_sync(FULL_MASK, e, o, LPR);
        const float v = __shfl_sync(FULL_MASK, d, o, LPR);
        all += eo == e ? v : 0.f;
      }
      d = all;
      if (e >= 0) mine[slot_of<S>(e)] = d;
      __syncwarp();
    }
    Tl* row_out = static_cast<Tl*>(g.out) + static_cast<long long>(t) * g.ld_out;
    const float K = lse - pa - dot;  // (softmax)
    // A row's sums that are not finite (+inf logits under a z loss, such
    // gradients from the caller) are for route_backward_row, which keeps them
    // from scores of 0.  The warp goes on there, since these rows are no common
    // ones: a choice between the two for every logit took 1 us of 33.  (Sums of
    // sigmoids are finite.)
    if (ROW && !SIGMOID && __any_sync(FULL_MASK, has && !(fabsf(K) < INFINITY))) break;
#pragma unroll
    for (int c = 0; c < S::C; ++c) {
      float o[S::CE];
      if (g.dgates) {
        load_cell_of<S>(mine, q, c, o);
      } else {
#pragma unroll
        for (int i = 0; i < S::CE; ++i) o[i] = 0.f;
      }
      if constexpr (ROW) {
        float a[S::CE];
        load_cell_of<S>(grad_smem, q, c, a);
#pragma unroll
        for (int i = 0; i < S::CE; ++i) {
          const int v = c * S::CE + i;
          if constexpr (SIGMOID) o[i] = fmaf(u[v] * inv * tt[v], a[i] - pa, o[i]);
          else o[i] = fmaf(u[v] * inv, a[i] + K, o[i]);
        }
        if constexpr (SIGMOID) {
          if (f.cz != 0.f) {
#pragma unroll
            for (int i = 0; i < S::CE; ++i) {
              const float v = unit_softmax(l[c * S::CE + i], m);
              if (v > 0.f) o[i] = fmaf(v, lse, o[i]);
            }
          }
        }
      }
      const int e0 = (c * LPR + q) * S::CE;
      if (g.wide_out) {
        if (has && e0 < N) store_cell<S::CE>(row_out + e0, o);
      } else {  // (a lane's own cell)
        store_cell_of<S>(mine, q, c, o);
      }
    }
    if (!g.wide_out) {
      // rows that are not aligned: through shared memory, so that neighbouring
      // lanes write neighbouring elements
      __syncwarp();
      for (int i = q; i < N; i += LPR) {
        const int at = slot_of<S>(i);
        if (has) row_out[i] = from_f32<Tl>(mine[at]);
        mine[at] = 0.f;
      }
      __syncwarp();
    }
    if (g.dgates && g.wide_out) {  // every lane has read its cells
      __syncwarp();
      if (e >= 0) mine[slot_of<S>(e)] = 0.f;
      __syncwarp();
    }
  }
  if constexpr (ROW && !SIGMOID) {
    if (t0 >= T) return;
    feed.drain(t0, step, T);
    for (; t0 < T; t0 += step)
      for (int t = t0; t < min(t0 + S::ROWS, T); ++t) route_backward_row(x, t, N, k, cfg, g, f, lane);
  }
}

// Rows of more experts than registers hold: a warp a row, several passes.
template <typename Tl>
__global__ __launch_bounds__(kGradWarps * 32) void route_backward_long_kernel(const __grid_constant__ Logits<Tl> x, int T,
                                                                              int N, int k,
                                                                              const __grid_constant__ RouteCfg cfg,
                                                                              const __grid_constant__ RouteGrad g) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const LossFactors f(g, N, k);
  for (int t = blockIdx.x * kGradWarps + w; t < T; t += gridDim.x * kGradWarps)
    route_backward_row(x, t, N, k, cfg, g, f, lane);
}

}  // namespace bfmoe
