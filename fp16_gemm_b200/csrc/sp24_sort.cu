// Token sort and unsort of the routed feed-forward: rows of x into expert order, expert outputs
// back in token order with the router weights applied, and the gradients of both (definitions in
// sp24.h; [P1] "Concurrency, not sparsity, is the lever" names the routed model).
//
// Everything here moves rows; nothing is multiplied more than once, so HBM is the bound.
#include "sp24_internal.cuh"

namespace sp24 {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kMaxUnsortTopk = 64;
constexpr int kCounters = 8192;  // counters of one pass over a chunk (32 KB of shared memory)

// ------------------------------------------------------------------ element access

template <int DT>
struct Elem;
template <>
struct Elem<SP24_F32> {
  using T = float;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float v) { return v; }
};
template <>
struct Elem<SP24_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<SP24_F16> {
  using T = __half;
  static __device__ __forceinline__ float get(T v) { return __half2float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
};

// V consecutive elements moved with one access.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

// ------------------------------------------------------------------ sort
//
// The row of entry i is the number of entries before it in the order (expert, entry number).  One
// warp finds it by counting and then moves the entry's row of x.
//
// Few entries: every warp counts over all of them, in one launch.  Many: the entries are cut into
// chunks of 2^chunk_log; a first launch counts each chunk's entries per expert (and all of them, by
// integer atomics, whose order does not matter), and the warp adds up the totals of lower experts, its
// expert's counts in earlier chunks and the equal entries before it in its own chunk.  Its reads grow
// like E + n / chunk + chunk instead of n, so the chunk is about sqrt(n).

struct SortTables {
  const int32_t* routing;
  int64_t n, E;
  int32_t *pos, *src, *row_expert, *offsets;
  const int32_t* counts;  // [E + 1][chunks]: by expert (E: the empty slots), then by chunk
  const int32_t* totals;  // [E + 1]
  int64_t chunks;
  int chunk_log;
};

// The expert of an entry; empty slots come after every expert.
__device__ __forceinline__ int64_t entry_key(int32_t id, int64_t E) { return id < 0 || id >= E ? E : id; }

template <bool MANY>
__device__ __forceinline__ int entries_below(const SortTables& t, int64_t key) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  if (MANY) {
    for (int64_t e = lane; e < key; e += 32) before += t.totals[e];
  } else {
    for (int64_t j = lane; j < t.n; j += 32) before += entry_key(t.routing[j], t.E) < key;
  }
  return before;
}

template <bool MANY>
__device__ __forceinline__ int equal_before(const SortTables& t, int64_t key, int64_t i) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  int64_t from = 0;
  if (MANY) {
    const int64_t chunk = i >> t.chunk_log;
    const int32_t* const mine = t.counts + key * t.chunks;
    for (int64_t c = lane; c < chunk; c += 32) before += mine[c];
    from = chunk << t.chunk_log;
  }
  for (int64_t j = from + lane; j < i; j += 32) before += entry_key(t.routing[j], t.E) == key;
  return before;
}

// One warp per entry, then one per offset.
template <int BYTES, bool MANY>
__global__ void __launch_bounds__(32 * kWarps) sort_kernel(const __grid_constant__ SortTables t,
                                                           const uint8_t* __restrict__ x, int topk, int64_t row_bytes,
                                                           uint8_t* __restrict__ xs) {
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= t.n + t.E + 1) return;
  if (i >= t.n) {
    const int at = __reduce_add_sync(kFull, entries_below<MANY>(t, i - t.n));
    if (lane == 0) t.offsets[i - t.n] = at;
    return;
  }
  const int32_t id = t.routing[i];
  const int64_t key = entry_key(id, t.E);
  const bool held = key < t.E;
  if (!held && id != -1 && lane == 0) set_dev_error(SP24_ERR_INVALID_ARG);
  const int row = __reduce_add_sync(kFull, entries_below<MANY>(t, key) + equal_before<MANY>(t, key, i));
  if (lane == 0) {
    t.pos[i] = held ? row : -1;
    t.src[row] = held ? (int32_t)i : -1;
    t.row_expert[row] = held ? id : -1;
  }
  if (!held || !x) return;
  using V = Vec<uint8_t, BYTES>;
  const V* from = reinterpret_cast<const V*>(x + (i / topk) * row_bytes);
  V* to = reinterpret_cast<V*>(xs + (int64_t)row * row_bytes);
  for (int64_t c = lane; c < row_bytes / BYTES; c += 32) to[c] = from[c];
}

// Each CTA counts one chunk; with E + 1 counters in shared memory.
__global__ void __launch_bounds__(256) sort_count_kernel(const int32_t* __restrict__ routing, int64_t n, int64_t E,
                                                         int chunk_log, int64_t chunks, int32_t* __restrict__ counts,
                                                         int32_t* __restrict__ totals) {
  extern __shared__ int32_t held[];
  const int64_t from = (int64_t)blockIdx.x << chunk_log, to = min(n, from + ((int64_t)1 << chunk_log));
  for (int64_t e0 = 0; e0 <= E; e0 += kCounters) {
    const int span = (int)min((int64_t)kCounters, E + 1 - e0);
    for (int e = threadIdx.x; e < span; e += 256) held[e] = 0;
    __syncthreads();
    for (int64_t j = from + threadIdx.x; j < to; j += 256) {
      const int64_t key = entry_key(routing[j], E) - e0;
      if (key >= 0 && key < span) atomicAdd(&held[key], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < span; e += 256) {
      const int32_t v = held[e];
      counts[(e0 + e) * chunks + blockIdx.x] = v;
      if (v) atomicAdd(&totals[e0 + e], v);
    }
    __syncthreads();
  }
}

// Above this many entries the chunked form is used: see sp24_moe_sort.
constexpr int64_t kFew = 2048;

struct SortWs {
  int chunk_log;
  int64_t chunks, totals_at, counts_at, bytes;
};

SortWs sort_layout(int64_t n, int64_t E) {
  SortWs w{};
  if (n <= kFew) return w;
  w.chunk_log = 8;
  while ((1ll << (2 * w.chunk_log)) < n) ++w.chunk_log;
  w.chunks = (n + (1ll << w.chunk_log) - 1) >> w.chunk_log;
  w.counts_at = ((E + 1) * 4 + 15) / 16 * 16;
  w.bytes = w.counts_at + (E + 1) * w.chunks * 4;
  return w;
}

// ------------------------------------------------------------------ unsort

// The row of entry i, or -1 for an empty slot.
__device__ __forceinline__ int entry_row(const int32_t* pos, int64_t i, int64_t rows) {
  const int r = pos[i];
  if (r >= 0 && r < rows) return r;
  if (r != -1) set_dev_error(SP24_ERR_INVALID_ARG);
  return -1;
}

// One thread per V columns of one token; the slots in order.
template <int YS, int Y, int V>
__global__ void __launch_bounds__(256) unsort_kernel(const void* __restrict__ ys_, const int32_t* __restrict__ pos,
                                                     const float* __restrict__ router_w, int64_t T, int topk,
                                                     int64_t rows, int64_t H, void* __restrict__ y_) {
  using VI = Vec<typename Elem<YS>::T, V>;
  using VO = Vec<typename Elem<Y>::T, V>;
  const VI* ys = reinterpret_cast<const VI*>(ys_);
  VO* y = reinterpret_cast<VO*>(y_);
  const int64_t HV = H / V, total = T * HV;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / HV, c = i - t * HV;
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
    for (int s = 0; s < topk; ++s) {
      const int r = entry_row(pos, t * topk + s, rows);
      if (r < 0) continue;
      const float w = router_w ? router_w[t * topk + s] : 1.0f;
      const VI v = ys[r * HV + c];
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] = fmaf(w, Elem<YS>::get(v.e[k]), acc[k]);
    }
    VO o;
#pragma unroll
    for (int k = 0; k < V; ++k) o.e[k] = Elem<Y>::put(acc[k]);
    y[i] = o;
  }
}

// One warp per entry: its row of dys, and the dot product that is its weight's gradient.
template <int YS, int Y, int V>
__global__ void __launch_bounds__(32 * kWarps) unsort_backward_kernel(
    const void* __restrict__ dy_, const void* __restrict__ ys_, const int32_t* __restrict__ pos,
    const float* __restrict__ router_w, int64_t n, int topk, int64_t rows, int64_t H, void* __restrict__ dys_,
    float* __restrict__ d_router_w) {
  using VI = Vec<typename Elem<YS>::T, V>;
  using VO = Vec<typename Elem<Y>::T, V>;
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= n) return;
  const int r = entry_row(pos, i, rows);
  if (r < 0) {
    if (d_router_w && lane == 0) d_router_w[i] = 0.0f;
    return;
  }
  const float w = router_w ? router_w[i] : 1.0f;
  const int64_t HV = H / V;
  const VO* dy = reinterpret_cast<const VO*>(dy_) + (i / topk) * HV;
  const VI* ys = reinterpret_cast<const VI*>(ys_) + r * HV;
  VI* dys = reinterpret_cast<VI*>(dys_) + r * HV;
  float dot = 0.0f;
  for (int64_t c = lane; c < HV; c += 32) {
    const VO g = dy[c];
    VI d;
    if (d_router_w) {
      const VI v = ys[c];
#pragma unroll
      for (int k = 0; k < V; ++k) dot = fmaf(Elem<Y>::get(g.e[k]), Elem<YS>::get(v.e[k]), dot);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) d.e[k] = Elem<YS>::put(w * Elem<Y>::get(g.e[k]));
    dys[c] = d;
  }
  if (d_router_w) {
#pragma unroll
    for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(kFull, dot, d);
    if (lane == 0) d_router_w[i] = dot;
  }
}

// Calls f(std::integral_constant-like tags) for the type pairs the header names; 0 if it names none.
template <int YS, int Y>
struct Pair {
  static constexpr int ys = YS, y = Y;
};
template <typename F>
int by_pair(int ys, int y, F f) {
  if (ys == SP24_F32) {
    if (y == SP24_F32) return f(Pair<SP24_F32, SP24_F32>{});
    if (y == SP24_BF16) return f(Pair<SP24_F32, SP24_BF16>{});
    return f(Pair<SP24_F32, SP24_F16>{});
  }
  if (ys == SP24_BF16) {
    if (y == SP24_BF16) return f(Pair<SP24_BF16, SP24_BF16>{});
    return f(Pair<SP24_BF16, SP24_F32>{});
  }
  if (y == SP24_F16) return f(Pair<SP24_F16, SP24_F16>{});
  return f(Pair<SP24_F16, SP24_F32>{});
}

// The largest vector (elements) that H and the pointers allow, 16 bytes of the narrower type at most.
int vec_elems(int64_t H, const void* a, int ea, const void* b, int eb, const void* c, int ec) {
  for (int v = 16 / (ea < eb ? ea : eb); v > 1; v /= 2)
    if (H % v == 0 && aligned(a, v * ea < 16 ? v * ea : 16) && aligned(b, v * eb < 16 ? v * eb : 16) &&
        aligned(c, v * ec < 16 ? v * ec : 16))
      return v;
  return 1;
}

int check_unsort(int ys_dtype, int y_dtype, int64_t T, int topk, int64_t rows, int64_t H) {
  if (!elem_bytes(ys_dtype) || !elem_bytes(y_dtype)) return SP24_ERR_DTYPE;
  if (ys_dtype != SP24_F32 && y_dtype != SP24_F32 && ys_dtype != y_dtype) return SP24_ERR_DTYPE;
  if (T < 0 || topk < 1 || rows < 0 || H < 0) return SP24_ERR_SHAPE;
  if (topk > kMaxUnsortTopk || T > INT32_MAX || rows > INT32_MAX || T * topk > INT32_MAX) return SP24_ERR_UNSUPPORTED;
  return SP24_OK;
}

}  // namespace
}  // namespace sp24

using namespace sp24;

extern "C" int sp24_moe_sort_workspace_size(int64_t T, int topk, int64_t E, int64_t* bytes) {
  if (!bytes) return SP24_ERR_INVALID_ARG;
  if (T < 0 || topk < 1 || E < 1) return SP24_ERR_SHAPE;
  if (E > (1 << 20) || T > INT32_MAX || T * topk > INT32_MAX) return SP24_ERR_UNSUPPORTED;
  *bytes = sort_layout(T * topk, E).bytes;
  return SP24_OK;
}

extern "C" int sp24_moe_sort(const void* x, int dtype, const int32_t* routing, int64_t T, int topk, int64_t E,
                             int64_t H, void* xs, int32_t* pos, int32_t* src, int32_t* row_expert, int32_t* offsets,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  const int eb = elem_bytes(dtype);
  if (!eb) return SP24_ERR_DTYPE;
  if (T < 0 || topk < 1 || E < 1 || H < 0) return SP24_ERR_SHAPE;
  if (E > (1 << 20) || T > INT32_MAX || T * topk > INT32_MAX) return SP24_ERR_UNSUPPORTED;
  const int64_t n = T * topk;
  if (!offsets || (n && (!routing || !pos || !src || !row_expert))) return SP24_ERR_INVALID_ARG;
  if (n && H && !x != !xs) return SP24_ERR_INVALID_ARG;
  if (!aligned(x, eb) || !aligned(xs, eb) || !aligned(routing, 4) || !aligned(pos, 4) || !aligned(src, 4) ||
      !aligned(row_expert, 4) || !aligned(offsets, 4))
    return SP24_ERR_ALIGN;
  const SortWs ws = sort_layout(n, E);
  if (ws.bytes && (!workspace || workspace_bytes < ws.bytes)) return SP24_ERR_WORKSPACE;
  if (ws.bytes && !aligned(workspace, 16)) return SP24_ERR_ALIGN;
  cudaStream_t s = as_stream(stream);
  SortTables t{routing, n, E, pos, src, row_expert, offsets, nullptr, nullptr, ws.chunks, ws.chunk_log};
  if (ws.bytes) {
    int32_t* totals = reinterpret_cast<int32_t*>(workspace);
    int32_t* counts = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(workspace) + ws.counts_at);
    if (cudaMemsetAsync(totals, 0, (size_t)(E + 1) * 4, s) != cudaSuccess) return SP24_ERR_CUDA;
    const int64_t counters = E + 1 < kCounters ? E + 1 : kCounters;
    sort_count_kernel<<<(unsigned)ws.chunks, 256, (size_t)counters * 4, s>>>(routing, n, E, ws.chunk_log, ws.chunks,
                                                                             counts, totals);
    const int st = launch_status();
    if (st) return st;
    t.totals = totals;
    t.counts = counts;
  }
  const int64_t row = H * eb;
  const unsigned ctas = (unsigned)((n + E + 1 + kWarps - 1) / kWarps);
  const uint8_t* from = H ? reinterpret_cast<const uint8_t*>(x) : nullptr;
  uint8_t* to = reinterpret_cast<uint8_t*>(xs);
  auto run = [&](auto bytes) {
    constexpr int B = decltype(bytes)::value;
    if (ws.bytes)
      sort_kernel<B, true><<<ctas, 32 * kWarps, 0, s>>>(t, from, topk, row, to);
    else
      sort_kernel<B, false><<<ctas, 32 * kWarps, 0, s>>>(t, from, topk, row, to);
    return launch_status();
  };
  if (row % 16 == 0 && aligned(x, 16) && aligned(xs, 16)) return run(std::integral_constant<int, 16>{});
  if (row % 4 == 0 && aligned(x, 4) && aligned(xs, 4)) return run(std::integral_constant<int, 4>{});
  return run(std::integral_constant<int, 2>{});
}

extern "C" int sp24_moe_unsort(const void* ys, int ys_dtype, const int32_t* pos, const float* router_w, int64_t T,
                               int topk, int64_t rows, int64_t H, void* y, int y_dtype, void* stream) {
  const int st = check_unsort(ys_dtype, y_dtype, T, topk, rows, H);
  if (st) return st;
  if (T == 0 || H == 0) return SP24_OK;
  if ((rows && !ys) || !pos || !y) return SP24_ERR_INVALID_ARG;
  const int ei = elem_bytes(ys_dtype), eo = elem_bytes(y_dtype);
  if (!aligned(ys, ei) || !aligned(y, eo) || !aligned(pos, 4) || !aligned(router_w, 4)) return SP24_ERR_ALIGN;
  const int v = vec_elems(H, ys, ei, y, eo, nullptr, ei);
  cudaStream_t s = as_stream(stream);
  return by_pair(ys_dtype, y_dtype, [&](auto p) {
    auto run = [&](auto vec) {
      constexpr int V = decltype(vec)::value;
      const int64_t blocks = (T * (H / V) + 255) / 256, cap = (int64_t)sm_count() * 64;
      unsort_kernel<decltype(p)::ys, decltype(p)::y, V><<<(unsigned)(blocks < cap ? blocks : cap), 256, 0, s>>>(
          ys, pos, router_w, T, topk, rows, H, y);
      return launch_status();
    };
    if (v == 8) return run(std::integral_constant<int, 8>{});
    if (v == 4) return run(std::integral_constant<int, 4>{});
    return v == 2 ? run(std::integral_constant<int, 2>{}) : run(std::integral_constant<int, 1>{});
  });
}

extern "C" int sp24_moe_unsort_backward(const void* dy, int y_dtype, const void* ys, int ys_dtype, const int32_t* pos,
                                        const float* router_w, int64_t T, int topk, int64_t rows, int64_t H, void* dys,
                                        float* d_router_w, void* stream) {
  const int st = check_unsort(ys_dtype, y_dtype, T, topk, rows, H);
  if (st) return st;
  if (T == 0) return SP24_OK;
  if (!pos || (H && (!dy || (rows && !dys) || (rows && d_router_w && !ys)))) return SP24_ERR_INVALID_ARG;
  const int ei = elem_bytes(ys_dtype), eo = elem_bytes(y_dtype);
  if (!aligned(ys, ei) || !aligned(dys, ei) || !aligned(dy, eo) || !aligned(pos, 4) || !aligned(router_w, 4) ||
      !aligned(d_router_w, 4))
    return SP24_ERR_ALIGN;
  const int v = vec_elems(H, ys, ei, dy, eo, dys, ei);
  cudaStream_t s = as_stream(stream);
  const int64_t n = T * topk;
  return by_pair(ys_dtype, y_dtype, [&](auto p) {
    auto run = [&](auto vec) {
      constexpr int V = decltype(vec)::value;
      unsort_backward_kernel<decltype(p)::ys, decltype(p)::y, V>
          <<<(unsigned)((n + kWarps - 1) / kWarps), 32 * kWarps, 0, s>>>(dy, ys, pos, router_w, n, topk, rows, H, dys,
                                                                         d_router_w);
      return launch_status();
    };
    if (v == 8) return run(std::integral_constant<int, 8>{});
    if (v == 4) return run(std::integral_constant<int, 4>{});
    return v == 2 ? run(std::integral_constant<int, 2>{}) : run(std::integral_constant<int, 1>{});
  });
}
