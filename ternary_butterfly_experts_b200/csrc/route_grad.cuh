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

// Sums of one row for the losses.
struct RowSums {
  float m, z, s;  // largest logit, sum of unit_softmax, sum of unit_sigmoid
};
template <typename Tl>
__device__ __forceinline__ RowSums row_sums(const Tl* row, int N, int lane, bool sigmoid) {
  RowSums r;
  float m = -INFINITY;
  for (int e = lane; e < N; e += 32) m = fmaxf(m, to_f32(row[e]));
  r.m = warp_max(m);
  const float low = fminf(r.m, 0.f);
  float z = 0.f, s = 0.f;
  for (int e = lane; e < N; e += 32) {
    const float l = to_f32(row[e]);
    if (masked_logit(l)) continue;
    z += unit_softmax(l, r.m);
    if (sigmoid) s += unit_sigmoid(l, low);
  }
  r.z = warp_sum(z);
  r.s = sigmoid ? warp_sum(s) : r.z;
  return r;
}

// Per-block sums of the losses' terms: part [grid][N] sums of p_te, zpart
// [grid] of lse^2, and the counts of chosen slots and of rows into load (zeroed).
template <typename Tl>
__global__ __launch_bounds__(kGradWarps * 32) void balance_rows_kernel(const Tl* __restrict__ logits, long long ld,
                                                                       int T, int N, int k, int score,
                                                                       const int32_t* __restrict__ idx,
                                                                       float* __restrict__ part,
                                                                       double* __restrict__ zpart,
                                                                       int32_t* __restrict__ load) {
  extern __shared__ float col[];  // [kGradWarps][N]
  __shared__ double zs[kGradWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float* mine = col + static_cast<size_t>(w) * N;
  for (int e = lane; e < N; e += 32) mine[e] = 0.f;
  const bool sig = score == BFMOE_SCORE_SIGMOID;
  double z2 = 0.0;
  int rows = 0;
  for (int t = blockIdx.x * kGradWarps + w; t < T; t += gridDim.x * kGradWarps) {
    const Tl* row = logits + static_cast<long long>(t) * ld;
    const RowSums r = row_sums(row, N, lane, sig);
    if (!(r.m > -INFINITY)) continue;
    const float low = fminf(r.m, 0.f), inv = 1.f / r.s;
    for (int e = lane; e < N; e += 32) {
      const float l = to_f32(row[e]);
      if (!masked_logit(l)) mine[e] += (sig ? unit_sigmoid(l, low) : unit_softmax(l, r.m)) * inv;
    }
    const double lse = static_cast<double>(r.m) + static_cast<double>(logf(r.z));
    z2 += lse * lse;
    ++rows;
    if (lane < k) {
      const int e = idx[static_cast<long long>(t) * k + lane];
      if (e >= 0 && e < N) atomicAdd(load + e, 1);
      else report_error(BFMOE_EDEVICE_BOUNDS, static_cast<unsigned>(t));
    }
  }
  if (lane == 0) {
    zs[w] = z2;
    if (rows) atomicAdd(load + N, rows);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < N; e += blockDim.x) {
    float s = 0.f;
    for (int q = 0; q < kGradWarps; ++q) s += col[static_cast<size_t>(q) * N + e];
    part[static_cast<size_t>(blockIdx.x) * N + e] = s;
  }
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int q = 0; q < kGradWarps; ++q) s += zs[q];
    zpart[blockIdx.x] = s;
  }
}

__global__ __launch_bounds__(1024) void balance_finish_kernel(const float* __restrict__ part,
                                                              const double* __restrict__ zpart, int blocks, int N,
                                                              int k, const int32_t* __restrict__ load,
                                                              float* __restrict__ loss) {
  __shared__ double red[32];
  double s = 0.0;
  for (int e = threadIdx.x; e < N; e += blockDim.x) {
    double p = 0.0;
    for (int b = 0; b < blocks; ++b) p += static_cast<double>(part[static_cast<size_t>(b) * N + e]);
    s += p * static_cast<double>(load[e]);
  }
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double b = 0.0, z = 0.0;
    for (int q = 0; q < static_cast<int>(blockDim.x) / 32; ++q) b += red[q];
    for (int q = 0; q < blocks; ++q) z += zpart[q];
    const double R = static_cast<double>(load[N]);
    loss[0] = R > 0.0 ? static_cast<float>(b * N / (static_cast<double>(k) * R * R)) : 0.f;
    loss[1] = R > 0.0 ? static_cast<float>(z / R) : 0.f;
  }
}

template <typename Tl>
__global__ __launch_bounds__(kGradWarps * 32) void route_backward_kernel(
    const Tl* logits, long long ld, int T, int N, int k, RouteCfg cfg, const int32_t* __restrict__ idx,
    const float* __restrict__ dgates, const int32_t* __restrict__ load, const float* __restrict__ dloss, Tl* dlogits,
    long long ldd) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const bool sig = cfg.score == BFMOE_SCORE_SIGMOID;
  const bool dense = dgates && !sig && !cfg.renorm;  // every logit moves every gate
  float cb = 0.f, cz = 0.f, fs = 0.f;
  if (load) {
    const float R = static_cast<float>(load[N]);
    if (R > 0.f) {
      cb = dloss[0] * static_cast<float>(N) / R;
      cz = 2.f * dloss[1] / R;
      fs = 1.f / (static_cast<float>(k) * R);
    }
  }
  for (int t = blockIdx.x * kGradWarps + w; t < T; t += gridDim.x * kGradWarps) {
    const Tl* row = logits + static_cast<long long>(t) * ld;
    Tl* out = dlogits + static_cast<long long>(t) * ldd;
    RowSums r{-INFINITY, 0.f, 0.f};
    if (load || dense) r = row_sums(row, N, lane, sig);
    const float low = fminf(r.m, 0.f);
    const float inv_z = r.z > 0.f ? 1.f / r.z : 0.f, inv_s = r.s > 0.f ? 1.f / r.s : 0.f;
    // the chosen: lane j < k holds slot j and its share of the gradient
    int e = -1;
    float d = 0.f, dense_sum = 0.f;
    if (dgates) {
      float l = -INFINITY, dg = 0.f;
      if (lane < k) {
        e = idx[static_cast<long long>(t) * k + lane];
        if (e < 0 || e >= N) {
          report_error(BFMOE_EDEVICE_BOUNDS, static_cast<unsigned>(t));
          e = -1;
        } else {
          l = to_f32(row[e]);
          dg = dgates[static_cast<long long>(t) * k + lane] * cfg.scale;
        }
      }
      const bool live = e >= 0 && !masked_logit(l);
      if (dense) {
        d = live ? unit_softmax(l, r.m) * inv_z * dg : 0.f;
        dense_sum = warp_sum(d);
      } else if (cfg.renorm) {
        const float m = warp_max(live ? l : -INFINITY);
        const float u = !live ? 0.f : (sig ? unit_sigmoid(l, fminf(m, 0.f)) : unit_softmax(l, m));
        const float s = warp_sum(u);
        const float q = s > 0.f ? u / s : 0.f;
        const float dot = warp_sum(q * dg);
        d = q * (dg - dot);
      } else {
        d = live ? dg * sigmoid_fast(l) : 0.f;
      }
      if (sig) d = live ? d * sigmoid_fast(-l) : 0.f;
    }
    float fp = 0.f;
    if (load && cb != 0.f) {
      for (int q = lane; q < N; q += 32) {
        const float l = to_f32(row[q]);
        if (masked_logit(l)) continue;
        fp += (sig ? unit_sigmoid(l, low) : unit_softmax(l, r.m)) * inv_s * (static_cast<float>(load[q]) * fs);
      }
      fp = warp_sum(fp);
    }
    const float lse = r.m + logf(r.z);
    __syncwarp();
    for (int q0 = 0; q0 < N; q0 += 32) {
      const int q = q0 + lane;
      float g = 0.f;
      if (q < N) {
        const float l = to_f32(row[q]);
        if (!masked_logit(l)) {
          const float p = load || dense ? unit_softmax(l, r.m) * inv_z : 0.f;
          if (dense) g -= p * dense_sum;
          if (cb != 0.f) {
            const float ps = sig ? unit_sigmoid(l, low) * inv_s : p;
            float b = cb * ps * (static_cast<float>(load[q]) * fs - fp);
            if (sig) b *= sigmoid_fast(-l);
            g += b;
          }
          if (cz != 0.f) g += cz * lse * p;
        }
      }
      for (int j = 0; j < k; ++j) {
        const int ej = __shfl_sync(FULL_MASK, e, j);
        const float dj = __shfl_sync(FULL_MASK, d, j);
        if (ej == q) g += dj;
      }
      if (q < N) out[q] = from_f32<Tl>(g);
    }
    __syncwarp();
  }
}

}  // namespace bfmoe
