// Host-side helpers shared by the translation units of libbfmoe.so: error
// text, launch accounting and tracing, per-device kernel attributes.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>
#include <utility>
#include <vector>

#include "bfmoe.h"

namespace bfmoe {

inline thread_local char g_last_error[512] = "";

inline int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return code;
}
inline int ok() {
  g_last_error[0] = '\0';
  return BFMOE_OK;
}
inline int cuda_fail(cudaError_t e, const char* what) {
  return fail(BFMOE_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool is_pow2(long long v) { return v > 0 && (v & (v - 1)) == 0; }
inline int ilog2(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline int words_per_row(int d) { return std::max(1, (d + 15) / 16); }

// ---------------------------------------------------------------------------
// Launch accounting and optional per-launch CUDA events.
// ---------------------------------------------------------------------------
inline std::atomic<unsigned long long> g_launches{0};
inline std::mutex g_prof_mu;
inline bool g_prof_on = false;
struct ProfRec {
  const char* name;
  cudaEvent_t a, b;
};
inline std::vector<ProfRec> g_prof;
inline std::vector<cudaEvent_t> g_event_pool;

inline cudaEvent_t pool_event() {
  if (!g_event_pool.empty()) {
    cudaEvent_t e = g_event_pool.back();
    g_event_pool.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  cudaEventCreate(&e);
  return e;
}

template <typename F>
cudaError_t launch(const char* name, cudaStream_t s, F&& f) {
  ProfRec rec{name, nullptr, nullptr};
  bool prof;
  {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    prof = g_prof_on;
    if (prof) {
      rec.a = pool_event();
      rec.b = pool_event();
    }
  }
  if (prof) cudaEventRecord(rec.a, s);
  f();
  const cudaError_t e = cudaGetLastError();
  if (prof) {
    cudaEventRecord(rec.b, s);
    std::lock_guard<std::mutex> lk(g_prof_mu);
    g_prof.push_back(rec);
  }
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return e;
}

// Launch with programmatic stream serialisation: the kernel may start while
// the previous kernel of the stream finishes; it waits for that kernel's
// results with pdl_wait() before touching global memory.
template <typename... KP, typename... A>
void pdl_launch(void (*kern)(KP...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...);
}

// Kernel attributes (dynamic shared-memory limits) are set per device: the
// first launch of a kernel on each device sets them.  `done` holds one bit
// per device and is set only after the attribute, so concurrent first calls
// both set it (the call is idempotent).
inline int current_device() {
  int dev = 0;
  cudaGetDevice(&dev);
  return dev & 63;
}
inline bool needs_attr(const std::atomic<uint64_t>& done) {
  return (done.load(std::memory_order_acquire) >> current_device() & 1u) == 0;
}
inline void attr_set(std::atomic<uint64_t>& done) {
  done.fetch_or(uint64_t(1) << current_device(), std::memory_order_release);
}

inline int grid_for(long long work, int per_block, int cap) {
  long long g = (work + per_block - 1) / per_block;
  if (g < 1) g = 1;
  if (g > cap) g = cap;
  return static_cast<int>(g);
}

// SMs of the current device (cached per device).
inline int sm_count() {
  static std::atomic<int> n[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  dev &= 63;
  int v = n[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    if (v <= 0) v = 148;
    n[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

inline int check_dtype(int xdt) {
  if (xdt != BFMOE_F32 && xdt != BFMOE_BF16) return fail(BFMOE_EINVAL, "x_dtype=%d is not BFMOE_F32 or BFMOE_BF16", xdt);
  return BFMOE_OK;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The buckets of the routed rows (bucket.cuh) from idx [R]: chunk histograms
// cc ([ceil(R / 128k)][N]; read when have_histograms, else counted here), the
// scan and the scatter.  totals [N] is scratch; pad_out may be NULL.
cudaError_t build_buckets(const int32_t* idx, long long R, int k, int N, bool have_histograms, int32_t* cc,
                          int32_t* totals, int32_t* counts, int32_t* offsets, int32_t* rows, int32_t* pad_out,
                          long long p_cap, cudaStream_t s);

// Reads and clears the device error word of route.cu's kernels (a
// __device__ variable belongs to one translation unit).
cudaError_t take_route_error(unsigned* code, unsigned* info);

}  // namespace bfmoe
