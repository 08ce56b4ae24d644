// Global norm of a list of gradients, and the list scaled to at most a given
// norm: norm = sqrt(sum of the squares of every element of every tensor),
// g' = g min(1, max_norm / norm).  Squares and their sum are float64, so that
// neither large nor small gradients leave the range and long sums lose
// nothing; the sums' order is fixed.  A norm that is not finite in float64
// (infinities or NaN among the elements) scales nothing.
//
// The list travels in the kernel's parameters (no copy to the device, nothing
// to keep alive for a captured graph): up to kGradsPerLaunch tensors a launch,
// or kGradsFew where they are enough (15 KB of parameters against 2).
#pragma once
#include "route.cuh"

namespace bfmoe {

// Streaming: a producer warp walks the list in chunks and copies each into a
// ring in shared memory (bulk copies), 16 consumer warps take them from there,
// so that loads are in flight while the list is searched and squares are
// summed.  One tensor: norm at 5.7 TB/s for 189 MB, 6.8 for 1.5 GB of float32
// (6.2 of bfloat16), bound by memory.  189 MB of bfloat16 in 144 tensors: norm
// 39 us, scaling 51 us (7.4 TB/s, part of it from L2).  (With
// loads into registers, 4 blocks of 512 threads an SM and four 16-byte loads a
// thread, the norm took 47 us: between a block's chunks nothing was in flight.)
constexpr int kGradsPerLaunch = 512;
constexpr int kGradsFew = 64;
constexpr int kGradConsumers = 512;
constexpr int kGradThreads = kGradConsumers + 32;
constexpr int kGradBlocks = 2;          // of an SM
// A chunk costs a block about 0.5 us besides its bytes: 189 MB of bfloat16 took
// 51 us in chunks of 16 KB, 43 us in chunks of 32 KB, the same in 48 KB.
constexpr int kGradChunkBytes = 32768;
constexpr int kGradStages = 3;          // chunks of a block on their way or in work
constexpr int kGradSmem = kGradStages * kGradChunkBytes;
constexpr int kGradMaxParts = 1024;     // partial sums of one call

// A tensor is cut at 16-byte boundaries: its first chunk has up to 15 bytes
// before the first one too (head elements), its last less than 16 bytes more.
template <int MAX>
struct GradListOf {
  const void* src[MAX];
  void* dst[MAX];
  long long len[MAX];
  int first[MAX + 1];  // chunks before each tensor
  uint8_t src_type[MAX], dst_type[MAX], head[MAX];
  int n;
};

inline int grad_head(const void* p, int type, long long len) {
  const int bytes = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15);
  return static_cast<int>(std::min<long long>(bytes / (type == BFMOE_BF16 ? 2 : 4), len));
}
inline long long grad_chunks(const void* p, int type, long long len) {
  const long long chunk = kGradChunkBytes / (type == BFMOE_BF16 ? 2 : 4);
  const long long body = len - grad_head(p, type, len);
  return std::max(1LL, body / chunk + (body % chunk != 0));
}

// The tensor of chunk c: the last i with first[i] <= c.
template <class G>
__device__ __forceinline__ int grad_of_chunk(const G& g, int c) {
  int lo = 0, hi = g.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Bytes at the end of the list that the norm leaves in L2 for the scaling, which
// begins there: what lies before is loaded to be replaced first.  (189 MB of
// bfloat16: 95.7 us without it, 92.5 with 48 MB, 90.5 with 80, 91.3 with 108.)
constexpr long long kGradKept = 80LL << 20;

__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void bulk_load_hint(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// A chunk of a tensor: `vecs` 16-byte vectors from element `at` on are in
// shared memory; `head` elements before `at` and `tail` behind them are not.
struct GradChunk {
  const void* src;
  void* dst;
  long long at;
  int vecs;
  uint8_t src_bf16, dst_bf16, head, tail;
};

// Chunks first, first + step, ... (count of them) through the ring.  The
// consumer threads call ready() once, while the first copies are on their way;
// where it says so use(chunk, vectors) for every chunk, else the copies stop
// there.  Chunks before `kept` are the first that L2 replaces.  Every wait is
// bounded; after one that ran out all return, the producer after its own copies.
template <class G, class R, class F>
__device__ __forceinline__ void grad_stream(const G& g, int first, int step, int count, int kept, R&& ready, F&& use) {
  extern __shared__ __align__(128) uint8_t grad_ring[];
  __shared__ uint64_t full[kGradStages], empty[kGradStages], go;
  __shared__ GradChunk meta[kGradStages];
  __shared__ int going;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kGradStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, kGradConsumers / 32);
    }
    mbar_init(&go, 1);
    mbar_fence_init();
  }
  __syncthreads();
  // chunk q goes through stage s for the turn-th time
  constexpr int stages = kGradStages;
  int s = 0, turn = 0;
  auto next = [&] {
    if (++s == stages) {
      s = 0;
      ++turn;
    }
  };
  if (threadIdx.x >= kGradConsumers) {
    if (threadIdx.x == kGradConsumers) {
      int q = 0;
      bool done = false;
      const uint64_t policy = evict_first_policy();
      // the tensor at hand: its list entry is read once
      int c0 = 0, c1 = 0, sh = 0, head = 0;
      long long len = 0;
      GradChunk m{};
      for (; q < count; ++q, next()) {
        const int c = first + q * step;
        if (c < c0 || c >= c1) {
          const int i = grad_of_chunk(g, c);
          c0 = g.first[i];
          c1 = g.first[i + 1];
          len = g.len[i];
          head = g.head[i];
          m.src = g.src[i];
          m.dst = g.dst[i];
          m.src_bf16 = g.src_type[i] == BFMOE_BF16;
          m.dst_bf16 = g.dst_type[i] == BFMOE_BF16;
          sh = m.src_bf16 ? 1 : 2;  // bytes of an element, as a shift
        }
        const int chunk = kGradChunkBytes >> sh;
        m.at = head + static_cast<long long>(c - c0) * chunk;
        const int n = static_cast<int>(min(len - m.at, static_cast<long long>(chunk)));
        m.vecs = n >> (4 - sh);
        m.head = static_cast<uint8_t>(c == c0 ? head : 0);
        m.tail = static_cast<uint8_t>(n - (m.vecs << (4 - sh)));
        if (q == stages) {
          done = mbar_wait(&go, 0, 0x2203u) ? !going : true;
          if (done) break;
        }
        if (turn > 0 && !mbar_wait(empty + s, (turn - 1) & 1, 0x2200u | s)) {
          done = true;
          break;
        }
        meta[s] = m;
        mbar_expect_tx(full + s, m.vecs * 16);
        if (m.vecs > 0) {
          void* to = grad_ring + s * kGradChunkBytes;
          const void* from = static_cast<const uint8_t*>(m.src) + (m.at << sh);
          if (c < kept) bulk_load_hint(to, from, m.vecs * 16, full + s, policy);
          else bulk_load(to, from, m.vecs * 16, full + s);
        }
      }
      // the copies in flight where nobody takes them any more
      if (q <= stages && !done) done = mbar_wait(&go, 0, 0x2204u) ? !going : true;
      if (done)
        for (int p = max(0, q - stages); p < q; ++p) mbar_wait(full + p % stages, (p / stages) & 1, 0x2201u);
    }
  } else {
    const bool on = ready();
    if (threadIdx.x == 0) {
      going = on;
      mbar_arrive(&go);
    }
    for (int q = 0; on && q < count; ++q, next()) {
      if (__any_sync(FULL_MASK, !mbar_wait(full + s, turn & 1, 0x2202u | s))) break;
      const GradChunk m = meta[s];
      use(m, reinterpret_cast<const uint4*>(grad_ring + s * kGradChunkBytes));
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(empty + s);
    }
  }
  __syncthreads();
}

// Sum over the consumer threads (or a block of as many); valid in warp 0.
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"r"(kGradConsumers) : "memory"); }
__device__ __forceinline__ double consumer_sum(double v, double* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  consumer_sync();
  return threadIdx.x < 32 ? warp_sum(threadIdx.x < kGradConsumers / 32 ? red[threadIdx.x] : 0.0) : 0.0;
}

// 16 bytes of a tensor as float32.
template <typename T>
constexpr int kGradVec = 16 / sizeof(T);
template <typename T>
__device__ __forceinline__ void grad_unpack(const uint4& u, float (&v)[kGradVec<T>]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(w[i]);
    } else {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ void add_square(double& s, float x) {
  const double v = static_cast<double>(x);
  s = fma(v, v, s);
}

// The squares of a vector.  (Making the float64 of a bfloat16 from its bits, to
// spare the conversion unit, which takes 16 a clock and SM: 34.8 us instead of
// 33.1 for one tensor of 189 MB, 242 instead of 245 for 1.5 GB.)
template <typename T>
__device__ __forceinline__ void square_vector(double (&s)[4], const uint4& u) {
  float f[kGradVec<T>];
  grad_unpack<T>(u, f);
#pragma unroll
  for (int q = 0; q < kGradVec<T>; ++q) add_square(s[q & 3], f[q]);
}

template <int MAX>
__global__ __launch_bounds__(kGradThreads, kGradBlocks) void grad_norm_kernel(const __grid_constant__ GradListOf<MAX> g,
                                                                              double* __restrict__ part) {
  __shared__ double red[32];
  pdl_wait();
  pdl_trigger();
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  const int chunks = g.first[g.n];
  const int mine = (chunks - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  const int kept = chunks - static_cast<int>(kGradKept / kGradChunkBytes);
  grad_stream(g, blockIdx.x, gridDim.x, mine, kept, [] { return true; }, [&](const GradChunk& m, const uint4* v) {
    const bool bf16 = m.src_bf16;
    if (bf16) {
#pragma unroll 4
      for (int i = threadIdx.x; i < m.vecs; i += kGradConsumers) square_vector<__nv_bfloat16>(s, v[i]);
    } else {
#pragma unroll 4
      for (int i = threadIdx.x; i < m.vecs; i += kGradConsumers) square_vector<float>(s, v[i]);
    }
    if (static_cast<int>(threadIdx.x) < m.head + m.tail) {
      const int r = threadIdx.x;
      const long long at = r < m.head ? r : m.at + static_cast<long long>(m.vecs) * (bf16 ? 8 : 4) + (r - m.head);
      add_square(s[0], bf16 ? to_f32(static_cast<const __nv_bfloat16*>(m.src)[at])
                            : static_cast<const float*>(m.src)[at]);
    }
  });
  if (threadIdx.x >= kGradConsumers) return;
  const double sum = consumer_sum((s[0] + s[1]) + (s[2] + s[3]), red);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__device__ __forceinline__ double grad_total(const double* __restrict__ part, int parts) {
  __shared__ double red[32];
  __shared__ double total;
  double s = 0.0;
  for (int q = threadIdx.x; q < parts; q += kGradConsumers) s += part[q];
  s = consumer_sum(s, red);
  if (threadIdx.x == 0) total = sqrt(s);
  consumer_sync();
  return total;
}

__global__ __launch_bounds__(kGradConsumers) void grad_norm_finish_kernel(const double* __restrict__ part, int parts,
                                                                        float* __restrict__ norm) {
  pdl_wait();
  pdl_trigger();
  const double v = grad_total(part, parts);
  if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

struct GradFactor {
  float first, by;  // applied one after the other
  bool on;
  __device__ __forceinline__ float operator()(float x) const { return on ? x * first * by : x; }
};

template <typename Td>
__device__ __forceinline__ void grad_store(Td* p, const float* v, int n) {
  if constexpr (sizeof(Td) == 4) {
#pragma unroll
    for (int q = 0; q < n; q += 4) __stcs(reinterpret_cast<float4*>(p + q), make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < n / 2; ++q) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
      w[q] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (n == 8) __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    else __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
  }
}

// A chunk from shared memory to d times f.  Wide where the output reaches a
// boundary together with the tensor (always when they are the same).
template <typename T, typename Td>
__device__ __forceinline__ void grad_scale_chunk(const GradChunk& m, const uint4* v, const T* p, Td* d, const GradFactor& f) {
  constexpr int VE = kGradVec<T>;
  constexpr size_t WANT = VE * sizeof(Td) < 16 ? VE * sizeof(Td) : 16;
  Td* out = d + m.at;
  if ((reinterpret_cast<uintptr_t>(out) & (WANT - 1)) == 0) {
#pragma unroll 4
    for (int i = threadIdx.x; i < m.vecs; i += kGradConsumers) {
      float x[VE];
      grad_unpack<T>(v[i], x);
#pragma unroll
      for (int q = 0; q < VE; ++q) x[q] = f(x[q]);
      grad_store(out + static_cast<size_t>(i) * VE, x, VE);
    }
  } else {
    const T* e = reinterpret_cast<const T*>(v);
    for (int i = threadIdx.x; i < m.vecs * VE; i += kGradConsumers) out[i] = from_f32<Td>(f(to_f32(e[i])));
  }
  if (static_cast<int>(threadIdx.x) < m.head + m.tail) {
    const int r = threadIdx.x;
    const long long at = r < m.head ? r : m.at + static_cast<long long>(m.vecs) * VE + (r - m.head);
    d[at] = from_f32<Td>(f(to_f32(p[at])));
  }
}

// The chunks are taken from the last one on: what the norm read last is still
// in L2.
template <int MAX>
__global__ __launch_bounds__(kGradThreads, kGradBlocks) void grad_scale_kernel(const __grid_constant__ GradListOf<MAX> g,
                                                                               const double* __restrict__ part,
                                                                               int parts, int all_in_place,
                                                                               float max_norm,
                                                                               float* __restrict__ norm) {
  // The copies start before the norm's kernel has ended: that kernel's blocks
  // had all seen the gradients' writers end, and it writes none itself.
  pdl_trigger();
  GradFactor f{};
  const int last = g.first[g.n] - 1 - static_cast<int>(blockIdx.x);
  grad_stream(g, last, -static_cast<int>(gridDim.x), last / static_cast<int>(gridDim.x) + 1, 0x7fffffff,
              [&] {
                pdl_wait();
                const double v = grad_total(part, parts);
                if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(v);
                f.on = v > static_cast<double>(max_norm) && v < INFINITY;
                // a factor below the normal float32 range is applied in two
                // steps, the first an exact power of two, to keep its 24 bits
                double by = static_cast<double>(max_norm) / v;
                f.first = by < 0x1p-100 ? 0x1p-80f : 1.f;
                if (by < 0x1p-100) by *= 0x1p80;
                f.by = static_cast<float>(by);
                return f.on || !all_in_place;
              },
              [&](const GradChunk& m, const uint4* vec) {
                const void* p = m.src;
                void* d = m.dst;
                if (!f.on && p == d) return;
                const bool to_bf16 = m.dst_bf16;
                if (m.src_bf16) {
                  const auto* x = static_cast<const __nv_bfloat16*>(p);
                  if (to_bf16) grad_scale_chunk(m, vec, x, static_cast<__nv_bfloat16*>(d), f);
                  else grad_scale_chunk(m, vec, x, static_cast<float*>(d), f);
                } else {
                  const auto* x = static_cast<const float*>(p);
                  if (to_bf16) grad_scale_chunk(m, vec, x, static_cast<__nv_bfloat16*>(d), f);
                  else grad_scale_chunk(m, vec, x, static_cast<float*>(d), f);
                }
              });
}

}  // namespace bfmoe
