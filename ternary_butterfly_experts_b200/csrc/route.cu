// Host side of routing from logits, its gradient, the balance losses and the
// gradient norm (include/bfmoe.h): argument checks, workspace layout, launches.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "common.cuh"
#include "grad_clip.cuh"
#include "host.cuh"
#include "route.cuh"
#include "route_grad.cuh"

namespace bfmoe {

cudaError_t take_route_error(unsigned* code, unsigned* info) {
  cudaError_t e = cudaMemcpyFromSymbol(code, g_err_code, sizeof(*code));
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(info, g_err_info, sizeof(*info));
  if (e != cudaSuccess || *code == 0) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbol(g_err_code, &zero, sizeof(zero));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_err_info, &zero, sizeof(zero));
  return e;
}

}  // namespace bfmoe

using namespace bfmoe;

namespace {

// Blocks of the loss kernel at most, which leaves one row of partial sums each.
constexpr int kBalanceBlocks = 640;

struct RoutePlan {
  size_t chunk_counts, totals;  // buckets
  size_t part, zpart, loads;    // balance loss
  size_t total;
};

RoutePlan make_route_plan(int N, long long T, int k) {
  RoutePlan p{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align_up(bytes, 256);
    return o;
  };
  const long long nchunks = std::max(1LL, (T + 127) / 128);
  (void)k;
  const size_t blocks = static_cast<size_t>(std::max(1LL, std::min<long long>(T, kBalanceBlocks)));
  p.chunk_counts = take(static_cast<size_t>(nchunks) * N * 4);
  p.totals = take(static_cast<size_t>(N) * 4);
  const size_t buckets_end = off;
  off = 0;
  p.part = take(blocks * N * 4);
  p.zpart = take(blocks * 8);
  p.loads = take(blocks * (N + 1) * 4);
  p.total = std::max(buckets_end, off);
  return p;
}

int check_routing_sizes(const char* what, int N, long long T, int k, long long ld, int dtype) {
  if (N < 1 || N > BFMOE_MAX_EXPERTS) return fail(BFMOE_EINVAL, "%s: n_experts=%d must be in [1, %d]", what, N, BFMOE_MAX_EXPERTS);
  if (k < 1 || k > BFMOE_MAX_K || k > N) return fail(BFMOE_EINVAL, "%s: k=%d must be in [1, min(%d, N=%d)]", what, k, BFMOE_MAX_K, N);
  if (T < 0) return fail(BFMOE_EINVAL, "%s: T=%lld must be >= 0", what, T);
  // (row ids, and the strides of grids over the rows, are int32)
  if (T * k > 0x7ff00000LL) return fail(BFMOE_EUNSUPPORTED, "%s: T*k=%lld exceeds int32 row ids", what, T * k);
  if (ld < N) return fail(BFMOE_EINVAL, "%s: row stride %lld is less than n_experts=%d", what, ld, N);
  if (dtype != BFMOE_F32 && dtype != BFMOE_BF16) return fail(BFMOE_EINVAL, "%s: dtype=%d is not BFMOE_F32 or BFMOE_BF16", what, dtype);
  return BFMOE_OK;
}

int check_scoring(const char* what, const bfmoe_scoring* s, int N, int k) {
  if (!s) return fail(BFMOE_EINVAL, "%s: NULL scoring", what);
  if (s->score != BFMOE_SCORE_SOFTMAX && s->score != BFMOE_SCORE_SIGMOID)
    return fail(BFMOE_EINVAL, "%s: score=%d is not softmax or sigmoid", what, s->score);
  if (s->group_score != BFMOE_GROUP_MAX && s->group_score != BFMOE_GROUP_TOP2)
    return fail(BFMOE_EINVAL, "%s: group_score=%d is not max or top2", what, s->group_score);
  if (s->n_groups < 1 || s->n_groups > BFMOE_MAX_GROUPS || N % s->n_groups != 0)
    return fail(BFMOE_EINVAL, "%s: n_groups=%d must divide n_experts=%d and be in [1, %d]", what, s->n_groups, N,
                BFMOE_MAX_GROUPS);
  if (s->top_groups < 1 || s->top_groups > s->n_groups)
    return fail(BFMOE_EINVAL, "%s: top_groups=%d must be in [1, n_groups=%d]", what, s->top_groups, s->n_groups);
  if (k > s->top_groups * (N / s->n_groups))
    return fail(BFMOE_EINVAL, "%s: k=%d exceeds the %d experts of the kept groups", what, k,
                s->top_groups * (N / s->n_groups));
  if (!std::isfinite(s->scale)) return fail(BFMOE_EINVAL, "%s: scale must be finite", what);
  return BFMOE_OK;
}

RouteCfg cfg_of(const bfmoe_scoring* s) {
  return RouteCfg{s->score, s->n_groups, s->top_groups, s->group_score, s->renormalize ? 1 : 0, s->scale};
}

int check_elem_align(const char* what, const char* name, const void* p, int dtype) {
  if (reinterpret_cast<uintptr_t>(p) & (dtype == BFMOE_BF16 ? 1u : 3u))
    return fail(BFMOE_EINVAL, "%s: %s must be aligned to its elements", what, name);
  return BFMOE_OK;
}

int check_space(const char* what, void* ws, size_t have, size_t need) {
  if (!ws) return fail(BFMOE_EWORKSPACE, "%s: workspace is NULL (%zu bytes needed)", what, need);
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(BFMOE_EWORKSPACE, "%s: workspace must be 256-byte aligned", what);
  if (have < need) return fail(BFMOE_EWORKSPACE, "%s: workspace has %zu bytes, %zu needed", what, have, need);
  return BFMOE_OK;
}

size_t type_size(int dtype) { return dtype == BFMOE_BF16 ? 2 : 4; }

int check_grads(const char* what, const bfmoe_grad* g, int n, bool with_out) {
  if (n < 0 || (n > 0 && !g)) return fail(BFMOE_EINVAL, "%s: n=%d tensors at %p", what, n, static_cast<const void*>(g));
  if (n > kGradsPerLaunch * 64) return fail(BFMOE_EUNSUPPORTED, "%s: more than %d tensors", what, kGradsPerLaunch * 64);
  for (int i = 0; i < n; ++i) {
    int rc;
    if (g[i].len < 0) return fail(BFMOE_EINVAL, "%s: tensor %d has length %lld", what, i, g[i].len);
    if ((g[i].dtype != BFMOE_F32 && g[i].dtype != BFMOE_BF16) ||
        (with_out && g[i].out && g[i].out_dtype != BFMOE_F32 && g[i].out_dtype != BFMOE_BF16))
      return fail(BFMOE_EINVAL, "%s: tensor %d is not BFMOE_F32 or BFMOE_BF16", what, i);
    if (g[i].len == 0) continue;
    if (!g[i].grad) return fail(BFMOE_EINVAL, "%s: tensor %d is NULL", what, i);
    if ((rc = check_elem_align(what, "a gradient", g[i].grad, g[i].dtype))) return rc;
    if (with_out && g[i].out) {
      if ((rc = check_elem_align(what, "an output", g[i].out, g[i].out_dtype))) return rc;
      if (g[i].out == g[i].grad && g[i].out_dtype != g[i].dtype)
        return fail(BFMOE_EINVAL, "%s: tensor %d is scaled in place into another type", what, i);
    }
  }
  return BFMOE_OK;
}

// What a clip writes may overlap nothing else of the list (a tensor scaled in
// place overlaps itself): an element must be read before it is written, once.
int check_overlap(const char* what, const bfmoe_grad* g, int n) {
  struct Span {
    uintptr_t a, b;
    int i;
    bool written;
  };
  try {
    std::vector<Span> v;
    v.reserve(static_cast<size_t>(n) * 2);
    for (int i = 0; i < n; ++i) {
      if (g[i].len == 0) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(g[i].grad);
      const bool in_place = !g[i].out || g[i].out == g[i].grad;
      v.push_back({a, a + static_cast<size_t>(g[i].len) * type_size(g[i].dtype), i, in_place});
      if (!in_place) {
        const uintptr_t o = reinterpret_cast<uintptr_t>(g[i].out);
        v.push_back({o, o + static_cast<size_t>(g[i].len) * type_size(g[i].out_dtype), i, true});
      }
    }
    std::sort(v.begin(), v.end(), [](const Span& x, const Span& y) { return x.a < y.a; });
    uintptr_t end = 0, end_written = 0;  // of all spans so far, of the written ones
    for (const Span& s : v) {
      if (s.a < end_written || (s.written && s.a < end))
        return fail(BFMOE_EINVAL, "%s: tensor %d overlaps memory that the call writes", what, s.i);
      end = std::max(end, s.b);
      if (s.written) end_written = std::max(end_written, s.b);
    }
  } catch (const std::bad_alloc&) {
    return fail(BFMOE_EINVAL, "%s: out of host memory for %d tensors", what, n);
  }
  return BFMOE_OK;
}

// Tensors [i0, i1) of the list as a kernel argument; empty ones are left out.
template <int MAX>
void fill_list(const bfmoe_grad* g, int i0, int i1, GradListOf<MAX>& out) {
  out.n = 0;
  long long chunks = 0;
  for (int i = i0; i < i1; ++i) {
    if (g[i].len == 0) continue;
    const int q = out.n++;
    out.src[q] = g[i].grad;
    out.dst[q] = g[i].out ? g[i].out : const_cast<void*>(static_cast<const void*>(g[i].grad));
    out.len[q] = g[i].len;
    out.src_type[q] = static_cast<uint8_t>(g[i].dtype);
    out.dst_type[q] = static_cast<uint8_t>(g[i].out ? g[i].out_dtype : g[i].dtype);
    out.first[q] = static_cast<int>(chunks);
    out.head[q] = static_cast<uint8_t>(grad_head(g[i].grad, g[i].dtype, g[i].len));
    chunks += grad_chunks(g[i].grad, g[i].dtype, g[i].len);
  }
  out.first[out.n] = static_cast<int>(chunks);
}

long long total_chunks(const bfmoe_grad* g, int n) {
  long long c = 0;
  for (int i = 0; i < n; ++i)
    if (g[i].len > 0) c += grad_chunks(g[i].grad, g[i].dtype, g[i].len);
  return c;
}

// The squares of the whole list into part; *parts: how many partial sums.
template <int MAX>
int launch_norm(const char* what, const bfmoe_grad* g, int n, double* part, int* parts, cudaStream_t s) {
  *parts = 0;
  static std::atomic<uint64_t> done{0};
  if (needs_attr(done)) {
    cudaError_t e = cudaFuncSetAttribute(grad_norm_kernel<MAX>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGradSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(grad_scale_kernel<MAX>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGradSmem);
    if (e != cudaSuccess) return cuda_fail(e, what);
    attr_set(done);
  }
  const int lists = (n + MAX - 1) / MAX;
  const int cap = lists ? std::min(sm_count() * kGradBlocks, kGradMaxParts / lists) : 0;
  GradListOf<MAX> l;
  for (int q = 0; q < lists; ++q) {
    fill_list(g, q * MAX, std::min(n, (q + 1) * MAX), l);
    if (l.first[l.n] == 0) continue;
    const int grid = std::min(l.first[l.n], cap);
    const cudaError_t e = launch("grad_norm", s, [&] {
      pdl_launch(grad_norm_kernel<MAX>, grid, kGradThreads, kGradSmem, s, l, part + *parts);
    });
    if (e != cudaSuccess) return cuda_fail(e, what);
    *parts += grid;
  }
  return BFMOE_OK;
}

// Norm, then scaling.  *written: whether the norm has been.
template <int MAX>
int launch_clip(const bfmoe_grad* g, int n, float max_norm, float* norm, double* part, int* parts, bool* written,
                cudaStream_t s) {
  int rc = launch_norm<MAX>("grad_clip: launch", g, n, part, parts, s);
  if (rc) return rc;
  GradListOf<MAX> l;
  for (int i0 = 0; i0 < n; i0 += MAX) {
    fill_list(g, i0, std::min(n, i0 + MAX), l);
    if (l.first[l.n] == 0) continue;
    int in_place = 1;
    for (int q = 0; q < l.n; ++q) in_place &= l.src[q] == l.dst[q];
    const int grid = std::min(l.first[l.n], sm_count() * kGradBlocks);
    float* out = *written ? nullptr : norm;  // once
    const cudaError_t e = launch("grad_scale", s, [&] {
      pdl_launch(grad_scale_kernel<MAX>, grid, kGradThreads, kGradSmem, s, l, static_cast<const double*>(part), *parts,
                 in_place, max_norm, out);
    });
    if (e != cudaSuccess) return cuda_fail(e, "grad_clip: launch");
    *written = true;
  }
  return BFMOE_OK;
}

// Calls f with the shape that rows of N <= 1024 experts take in the gradient
// and the losses: as few lanes a row as hold it at 16 logits a lane, since what
// a row takes besides its logits (sums over lanes, the chosen experts) is then
// shared by 2 or 4 rows of a warp.  65536 x 256 gradients: 38 us with 32 lanes
// of 8 logits.
template <class F>
cudaError_t with_shape(int N, bool cells, F&& f) {
  if (N <= 64) return f(RowShape<8, 8>{});
  if (!cells && N <= 128) return f(RowShape<16, 8>{});
  if (!cells && N <= 256) return f(RowShape<32, 8>{});
  if (N <= 128) return f(RowShape<8, 16>{});
  if (N <= 256) return f(RowShape<16, 16>{});
  if (N <= 512) return f(RowShape<32, 16>{});
  return f(RowShape<32, 32>{});
}

template <class S, int BY, bool GROUPED, typename Tl>
cudaError_t launch_route_rows(Logits<Tl> x, int T, int N, int k, const RouteCfg& cfg, const float* bias, int32_t* idx,
                              float* gates, cudaStream_t s) {
  // 1 << lsh lanes take a group: those that hold it where that is a power of
  // two, else as many as there are
  int lsh = 0;
  while (GROUPED && (2 << lsh) * cfg.n_groups <= 32) ++lsh;
  if (GROUPED && N % (cfg.n_groups * S::CE) == 0 && is_pow2(N / (cfg.n_groups * S::CE)) && S::C == 1)
    lsh = ilog2(N / (cfg.n_groups * S::CE));
  x.wide = wide_rows<S>(x.p, x.ld, N);
  const size_t floats = (BY != kByLogit ? S::MAXN : 0) + (GROUPED ? kRouteWarps * kGroupSpace<S> : 0) +
                        kRouteWarps * RowFeed<S, Tl>::bytes(x.wide) / 4;
  {
    static std::atomic<uint64_t> done{0};
    if (needs_attr(done)) {
      const cudaError_t e = cudaFuncSetAttribute(route_fast_kernel<S, Tl, BY, GROUPED>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 S::MAXN * 4 + kRouteWarps * (kGroupSpace<S> * 4 +
                                                                std::max(RowFeed<S, Tl>::bytes(true),
                                                                         RowFeed<S, Tl>::bytes(false))));
      if (e != cudaSuccess) return e;
      attr_set(done);
    }
  }
  const int grid = grid_for(T, kRouteWarps, sm_count() * kRouteBlocks<S>);
  return launch("route", s, [&] {
    pdl_launch(route_fast_kernel<S, Tl, BY, GROUPED>, grid, kRouteWarps * 32, floats * sizeof(float), s, x, T, N, k, cfg, bias,
               lsh, idx, gates);
  });
}

template <class S, typename Tl>
cudaError_t launch_route_shape(const Logits<Tl>& x, int T, int N, int k, const RouteCfg& cfg, const float* bias,
                               int32_t* idx, float* gates, cudaStream_t s) {
  const bool grouped = cfg.top_groups < cfg.n_groups;
  if (!bias && !(grouped && cfg.group_score == BFMOE_GROUP_TOP2)) {
    if (grouped) return launch_route_rows<S, kByLogit, true>(x, T, N, k, cfg, bias, idx, gates, s);
    return launch_route_rows<S, kByLogit, false>(x, T, N, k, cfg, bias, idx, gates, s);
  }
  if (cfg.score == BFMOE_SCORE_SOFTMAX) {
    if (grouped) return launch_route_rows<S, kBySoftmax, true>(x, T, N, k, cfg, bias, idx, gates, s);
    return launch_route_rows<S, kBySoftmax, false>(x, T, N, k, cfg, bias, idx, gates, s);
  }
  if (grouped) return launch_route_rows<S, kBySigmoid, true>(x, T, N, k, cfg, bias, idx, gates, s);
  return launch_route_rows<S, kBySigmoid, false>(x, T, N, k, cfg, bias, idx, gates, s);
}

// A row's logits in the registers of a warp up to 1024 experts.
template <typename Tl>
cudaError_t launch_route(const Logits<Tl>& x, int T, int N, int k, const RouteCfg& cfg, const float* bias, int32_t* idx,
                         float* gates, cudaStream_t s) {
  if (N <= 64) return launch_route_shape<RowShape<32, 2>>(x, T, N, k, cfg, bias, idx, gates, s);
  if (N <= 128) return launch_route_shape<RowShape<32, 4>>(x, T, N, k, cfg, bias, idx, gates, s);
  if (N <= 256) return launch_route_shape<RowShape<32, 8>>(x, T, N, k, cfg, bias, idx, gates, s);
  if (N <= 512) return launch_route_shape<RowShape<32, 16>>(x, T, N, k, cfg, bias, idx, gates, s);
  if (N <= 1024) return launch_route_shape<RowShape<32, 32>>(x, T, N, k, cfg, bias, idx, gates, s);
  return launch("route", s, [&] {
    pdl_launch(route_long_kernel<Tl>, grid_for(T, kRouteWarps, sm_count() * 8), kRouteWarps * 32, 0, s, x, T, N, k, cfg, bias,
               idx, gates);
  });
}

template <class S, bool SIGMOID, typename Tl>
cudaError_t launch_balance_rows(Logits<Tl> x, int T, int N, int k, const int32_t* idx, float* part, double* zpart,
                                int32_t* loads, int* grid, cudaStream_t s) {
  constexpr int feed = std::max(RowFeed<S, Tl>::bytes(true), RowFeed<S, Tl>::bytes(false));
  constexpr size_t most = kGradWarps * std::max(S::MAXN * 4, feed);
  const auto kern = balance_rows_kernel<S, Tl, SIGMOID>;
  static std::atomic<uint64_t> done{0};
  if (needs_attr(done)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) return e;
    attr_set(done);
  }
  x.wide = wide_rows<S>(x.p, x.ld, N);
  // a warp takes several rows where there are enough, so that the sums that
  // are left to add up stay few
  *grid = grid_for(T, kGradWarps * S::ROWS * 2, std::min(kBalanceBlocks, sm_count() * kBalanceRowBlocks<S>));
  return launch("balance_rows", s, [&] {
    pdl_launch(kern, *grid, kGradWarps * 32, most, s, x, T, N, k, idx, part, zpart, loads);
  });
}

template <typename Tl>
cudaError_t launch_balance(const Logits<Tl>& x, int T, int N, int k, bool sigmoid, const int32_t* idx, float* part, double* zpart,
                           int32_t* loads, int* grid, cudaStream_t s) {
  if (N <= 1024)
    return with_shape(N, wide_rows<RowShape<32, 8>>(x.p, x.ld, N), [&](auto shape) {
      using S = decltype(shape);
      if (sigmoid) return launch_balance_rows<S, true>(x, T, N, k, idx, part, zpart, loads, grid, s);
      return launch_balance_rows<S, false>(x, T, N, k, idx, part, zpart, loads, grid, s);
    });
  static std::atomic<uint64_t> done{0};
  if (needs_attr(done)) {
    const cudaError_t e = cudaFuncSetAttribute(balance_long_kernel<Tl>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (kGradWarps + 1) * BFMOE_MAX_EXPERTS * 4);
    if (e != cudaSuccess) return e;
    attr_set(done);
  }
  *grid = grid_for(T, kGradWarps, std::min(kBalanceBlocks, sm_count() * 2));
  return launch("balance_rows", s, [&] {
    pdl_launch(balance_long_kernel<Tl>, *grid, kGradWarps * 32, static_cast<size_t>(kGradWarps + 1) * N * 4, s, x, T, N, k,
               sigmoid ? 1 : 0, idx, part, zpart, loads);
  });
}

template <class S, bool SIGMOID, bool ROW, typename Tl>
cudaError_t launch_backward_rows(Logits<Tl> x, int T, int N, int k, const RouteCfg& cfg, RouteGrad g, cudaStream_t s) {
  constexpr size_t base = S::MAXN * (1 + kGradWarps * S::ROWS) * 4;
  constexpr size_t most = base + kGradWarps * std::max(RowFeed<S, Tl>::bytes(true), RowFeed<S, Tl>::bytes(false));
  const auto kern = route_backward_kernel<S, Tl, SIGMOID, ROW>;
  static std::atomic<uint64_t> done{0};
  if (needs_attr(done)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) return e;
    attr_set(done);
  }
  x.wide = wide_rows<S>(x.p, x.ld, N);
  g.wide_out = wide_rows<S>(static_cast<const Tl*>(g.out), g.ld_out, N);
  const int grid = grid_for(T, kGradWarps * S::ROWS, sm_count() * (ROW ? kGradRowBlocks<S> : 4));
  return launch("route_backward", s, [&] {
    pdl_launch(kern, grid, kGradWarps * 32, base + (ROW ? kGradWarps * RowFeed<S, Tl>::bytes(x.wide) : 0), s, x, T, N, k, cfg, g);
  });
}

template <typename Tl>
cudaError_t launch_route_backward(const Logits<Tl>& x, int T, int N, int k, const RouteCfg& cfg, const RouteGrad& g,
                                  cudaStream_t s) {
  if (N <= 1024)
    return with_shape(N, wide_rows<RowShape<32, 8>>(x.p, x.ld, N), [&](auto shape) {
      using S = decltype(shape);
      const bool sigmoid = cfg.score == BFMOE_SCORE_SIGMOID;
      // losses, and gates that are a softmax of the whole row, reach every logit
      if (!g.load && (sigmoid || cfg.renorm)) {
        if (sigmoid) return launch_backward_rows<S, true, false>(x, T, N, k, cfg, g, s);
        return launch_backward_rows<S, false, false>(x, T, N, k, cfg, g, s);
      }
      if (sigmoid) return launch_backward_rows<S, true, true>(x, T, N, k, cfg, g, s);
      return launch_backward_rows<S, false, true>(x, T, N, k, cfg, g, s);
    });
  return launch("route_backward", s, [&] {
    pdl_launch(route_backward_long_kernel<Tl>, grid_for(T, kGradWarps, sm_count() * 8), kGradWarps * 32, 0, s, x, T, N, k,
               cfg, g);
  });
}

}  // namespace

extern "C" {

size_t bfmoe_route_workspace_size(int n_experts, int T, int k) {
  if (check_routing_sizes("route_workspace_size", n_experts, T, k, n_experts, BFMOE_F32) != BFMOE_OK) return 0;
  return make_route_plan(n_experts, T, k).total;
}

int bfmoe_route(const void* logits, int dtype, int T, long long ld, int n_experts, int k, const bfmoe_scoring* scoring,
                const float* balance_bias, int32_t* idx, float* gates, int32_t* counts, int32_t* offsets,
                int32_t* rows, void* ws, size_t ws_bytes, bfmoe_stream_t stream) {
  const int N = n_experts;
  int rc = check_routing_sizes("route", N, T, k, ld, dtype);
  if (rc || (rc = check_scoring("route", scoring, N, k))) return rc;
  const bool buckets = counts || offsets || rows;
  if (buckets && (!counts || !offsets || (!rows && T > 0)))
    return fail(BFMOE_EINVAL, "route: counts, offsets and rows must be all given or all NULL");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (T == 0) {
    if (!buckets) return ok();
    if ((e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * N, s)) != cudaSuccess ||
        (e = cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (N + 1), s)) != cudaSuccess)
      return cuda_fail(e, "route: memset");
    return ok();
  }
  if (!logits || !idx || !gates) return fail(BFMOE_EINVAL, "route: NULL pointer");
  if ((rc = check_elem_align("route", "logits", logits, dtype))) return rc;
  const RoutePlan p = make_route_plan(N, T, k);
  if (buckets && (rc = check_space("route", ws, ws_bytes, p.total))) return rc;
  const RouteCfg cfg = cfg_of(scoring);
  e = dtype == BFMOE_BF16
          ? launch_route(Logits<__nv_bfloat16>{static_cast<const __nv_bfloat16*>(logits), ld, 0}, T, N, k, cfg,
                         balance_bias, idx, gates, s)
          : launch_route(Logits<float>{static_cast<const float*>(logits), ld, 0}, T, N, k, cfg, balance_bias, idx,
                         gates, s);
  if (e != cudaSuccess) return cuda_fail(e, "route: launch");
  if (!buckets) return ok();
  uint8_t* W = static_cast<uint8_t*>(ws);
  e = build_buckets(idx, static_cast<long long>(T) * k, k, N, false, reinterpret_cast<int32_t*>(W + p.chunk_counts),
                    reinterpret_cast<int32_t*>(W + p.totals), counts, offsets, rows, nullptr, 0, s);
  if (e != cudaSuccess) return cuda_fail(e, "route: buckets");
  return ok();
}

int bfmoe_balance_loss(const void* logits, int dtype, int T, long long ld, int n_experts, int k, int score,
                       const int32_t* idx, float* loss, int32_t* load, void* ws, size_t ws_bytes,
                       bfmoe_stream_t stream) {
  const int N = n_experts;
  int rc = check_routing_sizes("balance_loss", N, T, k, ld, dtype);
  if (rc) return rc;
  if (score != BFMOE_SCORE_SOFTMAX && score != BFMOE_SCORE_SIGMOID)
    return fail(BFMOE_EINVAL, "balance_loss: score=%d is not softmax or sigmoid", score);
  if (!loss || !load || (T > 0 && (!logits || !idx))) return fail(BFMOE_EINVAL, "balance_loss: NULL pointer");
  if ((rc = check_elem_align("balance_loss", "logits", logits, dtype))) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (T == 0) {
    if ((e = cudaMemsetAsync(load, 0, sizeof(int32_t) * (N + 1), s)) != cudaSuccess ||
        (e = cudaMemsetAsync(loss, 0, 2 * sizeof(float), s)) != cudaSuccess)
      return cuda_fail(e, "balance_loss: memset");
    return ok();
  }
  const RoutePlan p = make_route_plan(N, T, k);
  if ((rc = check_space("balance_loss", ws, ws_bytes, p.total))) return rc;
  uint8_t* W = static_cast<uint8_t*>(ws);
  float* part = reinterpret_cast<float*>(W + p.part);
  double* zpart = reinterpret_cast<double*>(W + p.zpart);
  int32_t* loads = reinterpret_cast<int32_t*>(W + p.loads);
  int grid = 0;
  const bool sigmoid = score == BFMOE_SCORE_SIGMOID;
  e = dtype == BFMOE_BF16
          ? launch_balance(Logits<__nv_bfloat16>{static_cast<const __nv_bfloat16*>(logits), ld, 0}, T, N, k, sigmoid,
                           idx, part, zpart, loads, &grid, s)
          : launch_balance(Logits<float>{static_cast<const float*>(logits), ld, 0}, T, N, k, sigmoid, idx, part, zpart,
                           loads, &grid, s);
  if (e != cudaSuccess) return cuda_fail(e, "balance_loss: launch");
  e = launch("balance_finish", s, [&] {
    pdl_launch(balance_finish_kernel, kFinishBlocks, kFinishThreads, 0, s, static_cast<const float*>(part),
               static_cast<const double*>(zpart), static_cast<const int32_t*>(loads), grid, N, k, load, loss);
  });
  if (e != cudaSuccess) return cuda_fail(e, "balance_loss: launch");
  return ok();
}

int bfmoe_route_backward(const void* logits, int dtype, int T, long long ld, int n_experts, int k,
                         const bfmoe_scoring* scoring, const float* balance_bias, const int32_t* idx,
                         const float* dgates, const int32_t* load, const float* dloss, void* dlogits,
                         long long ld_dlogits, bfmoe_stream_t stream) {
  const int N = n_experts;
  int rc = check_routing_sizes("route_backward", N, T, k, ld, dtype);
  if (rc || (rc = check_scoring("route_backward", scoring, N, k))) return rc;
  if (ld_dlogits < N) return fail(BFMOE_EINVAL, "route_backward: row stride %lld of dlogits is less than n_experts=%d", ld_dlogits, N);
  if ((load == nullptr) != (dloss == nullptr)) return fail(BFMOE_EINVAL, "route_backward: load and dloss must both be given or both NULL");
  if (T == 0) return ok();
  if (!logits || !dlogits || (dgates && !idx)) return fail(BFMOE_EINVAL, "route_backward: NULL pointer");
  if ((rc = check_elem_align("route_backward", "logits", logits, dtype)) ||
      (rc = check_elem_align("route_backward", "dlogits", dlogits, dtype)))
    return rc;
  if (logits == dlogits && ld != ld_dlogits) return fail(BFMOE_EINVAL, "route_backward: in place with another row stride");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const RouteCfg cfg = cfg_of(scoring);
  const RouteGrad g{idx, balance_bias, dgates, load, dloss, dlogits, ld_dlogits, 0};
  const cudaError_t e =
      dtype == BFMOE_BF16
          ? launch_route_backward(Logits<__nv_bfloat16>{static_cast<const __nv_bfloat16*>(logits), ld, 0}, T, N, k, cfg, g, s)
          : launch_route_backward(Logits<float>{static_cast<const float*>(logits), ld, 0}, T, N, k, cfg, g, s);
  if (e != cudaSuccess) return cuda_fail(e, "route_backward: launch");
  return ok();
}

size_t bfmoe_grad_workspace_size(void) { return kGradMaxParts * sizeof(double); }

int bfmoe_grad_norm(const bfmoe_grad* grads, int n, float* norm, void* ws, size_t ws_bytes, bfmoe_stream_t stream) {
  int rc = check_grads("grad_norm", grads, n, false);
  if (rc) return rc;
  if (!norm) return fail(BFMOE_EINVAL, "grad_norm: NULL norm");
  if (total_chunks(grads, n) > 0x7fffffffLL) return fail(BFMOE_EUNSUPPORTED, "grad_norm: too many elements");
  if ((rc = check_space("grad_norm", ws, ws_bytes, bfmoe_grad_workspace_size()))) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(ws);
  int parts = 0;
  rc = n <= kGradsFew ? launch_norm<kGradsFew>("grad_norm: launch", grads, n, part, &parts, s)
                      : launch_norm<kGradsPerLaunch>("grad_norm: launch", grads, n, part, &parts, s);
  if (rc) return rc;
  const cudaError_t e = launch("grad_norm_finish", s, [&] { pdl_launch(grad_norm_finish_kernel, 1, kGradConsumers, 0, s, part, parts, norm); });
  if (e != cudaSuccess) return cuda_fail(e, "grad_norm: launch");
  return ok();
}

int bfmoe_grad_clip(const bfmoe_grad* grads, int n, float max_norm, float* norm, void* ws, size_t ws_bytes,
                    bfmoe_stream_t stream) {
  int rc = check_grads("grad_clip", grads, n, true);
  if (rc) return rc;
  if (!norm) return fail(BFMOE_EINVAL, "grad_clip: NULL norm");
  if (!(max_norm >= 0.f)) return fail(BFMOE_EINVAL, "grad_clip: max_norm must be >= 0");
  if (total_chunks(grads, n) > 0x7fffffffLL) return fail(BFMOE_EUNSUPPORTED, "grad_clip: too many elements");
  if ((rc = check_overlap("grad_clip", grads, n))) return rc;
  if ((rc = check_space("grad_clip", ws, ws_bytes, bfmoe_grad_workspace_size()))) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(ws);
  int parts = 0;
  bool written = false;
  rc = n <= kGradsFew ? launch_clip<kGradsFew>(grads, n, max_norm, norm, part, &parts, &written, s)
                      : launch_clip<kGradsPerLaunch>(grads, n, max_norm, norm, part, &parts, &written, s);
  if (rc) return rc;
  if (!written) {  // nothing to scale: the norm of an empty list
    const cudaError_t e = launch("grad_norm_finish", s, [&] {
      pdl_launch(grad_norm_finish_kernel, 1, kGradConsumers, 0, s, static_cast<const double*>(part), parts, norm);
    });
    if (e != cudaSuccess) return cuda_fail(e, "grad_clip: launch");
  }
  return ok();
}

}  // extern "C"
