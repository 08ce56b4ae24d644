// Global norm of a list of gradients, and the list scaled to at most a given
// norm: norm = sqrt(sum of the squares of every element of every tensor),
// g' = g min(1, max_norm / norm).  Squares and their sum are float64, so that
// neither large nor small gradients leave the range and long sums lose
// nothing; the sums' order is fixed.  A norm that is not finite scales nothing.
//
// The list travels in the kernel's parameters (no copy to the device, nothing
// to keep alive for a captured graph): kGradsPerLaunch tensors a launch.
#pragma once
#include "route.cuh"

namespace bfmoe {

constexpr int kGradsPerLaunch = 512;
constexpr int kGradThreads = 512;
constexpr int kGradChunk = 8192;      // elements of a block's step
constexpr int kGradMaxParts = 1024;   // partial sums of one call

struct GradList {
  const void* src[kGradsPerLaunch];
  void* dst[kGradsPerLaunch];
  long long len[kGradsPerLaunch];
  int first[kGradsPerLaunch + 1];  // chunks before each tensor
  uint8_t src_type[kGradsPerLaunch], dst_type[kGradsPerLaunch];
  int n;
};

// The tensor of chunk c: the last i with first[i] <= c.
__device__ __forceinline__ int grad_of_chunk(const GradList& g, int c) {
  int lo = 0, hi = g.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v, double* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x < 32) {
    s = threadIdx.x < blockDim.x / 32 ? red[threadIdx.x] : 0.0;
    s = warp_sum(s);
  }
  return s;  // valid in warp 0
}

__device__ __forceinline__ float grad_load(const void* p, int type, long long i) {
  return type == BFMOE_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

__global__ __launch_bounds__(kGradThreads) void grad_norm_kernel(const __grid_constant__ GradList g,
                                                                 double* __restrict__ part) {
  __shared__ double red[32];
  double s = 0.0;
  const int chunks = g.first[g.n];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = grad_of_chunk(g, c);
    const long long a = static_cast<long long>(c - g.first[i]) * kGradChunk;
    const long long b = min(a + kGradChunk, g.len[i]);
    for (long long q = a + threadIdx.x; q < b; q += blockDim.x) {
      const double v = static_cast<double>(grad_load(g.src[i], g.src_type[i], q));
      s += v * v;
    }
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ double grad_total(const double* __restrict__ part, int parts) {
  __shared__ double red[32];
  __shared__ double total;
  double s = 0.0;
  for (int q = threadIdx.x; q < parts; q += blockDim.x) s += part[q];
  s = block_sum(s, red);
  if (threadIdx.x == 0) total = sqrt(s);
  __syncthreads();
  return total;
}

__global__ __launch_bounds__(kGradThreads) void grad_norm_finish_kernel(const double* __restrict__ part, int parts,
                                                                        float* __restrict__ norm) {
  const double v = grad_total(part, parts);
  if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

__global__ __launch_bounds__(kGradThreads) void grad_scale_kernel(const __grid_constant__ GradList g,
                                                                  const double* __restrict__ part, int parts,
                                                                  float max_norm, float* __restrict__ norm) {
  const double v = grad_total(part, parts);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(v);
  const bool clip = v > static_cast<double>(max_norm) && v < INFINITY;
  // a factor below the normal float32 range is applied in two steps, the
  // first an exact power of two, so that it keeps its 24 bits
  double f = static_cast<double>(max_norm) / v;
  const float first = f < 0x1p-100 ? 0x1p-80f : 1.f;
  if (f < 0x1p-100) f *= 0x1p80;
  const float by = clip ? static_cast<float>(f) : 1.f;
  const int chunks = g.first[g.n];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = grad_of_chunk(g, c);
    if (!clip && g.src[i] == g.dst[i]) continue;
    const long long a = static_cast<long long>(c - g.first[i]) * kGradChunk;
    const long long b = min(a + kGradChunk, g.len[i]);
    for (long long q = a + threadIdx.x; q < b; q += blockDim.x) {
      const float x = grad_load(g.src[i], g.src_type[i], q);
      const float y = clip ? x * first * by : x;
      if (g.dst_type[i] == BFMOE_BF16) static_cast<__nv_bfloat16*>(g.dst[i])[q] = __float2bfloat16_rn(y);
      else static_cast<float*>(g.dst[i])[q] = y;
    }
  }
}

}  // namespace bfmoe
