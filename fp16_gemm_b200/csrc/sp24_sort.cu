// Token sort and unsort of the routed feed-forward: rows of x into expert order, expert outputs
// back in token order with the router weights applied, and the gradients of both (definitions in
// sp24.h; [P1] "Concurrency, not sparsity, is the lever" names the routed model).
//
// Everything here moves rows; nothing is multiplied more than once, so HBM is the bound.  Measured at
// 4096 tokens x 10 slots, rows of 2048 bf16 entries (185 MB moved one way, 28 us at the copy rate): sort 34 us,
// its gradient 27 us, unsort 28 us, its gradients 57 us (354 MB, 54 us).  A decode step (8 tokens): about 3 us
// each, the time of a launch and two dependent loads.
#include "sp24_launch.cuh"

namespace sp24 {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kMaxUnsortTopk = 64;
constexpr int kCounters = 8192;  // counters of one pass over a chunk (32 KB of shared memory)

// ------------------------------------------------------------------ element access

// V consecutive elements of type DT as 32-bit words (one half word for a single 16-bit element), moved
// with accesses of at most 16 bytes, whatever the vector's size.
template <int BYTES>
struct Words {
  uint32_t w[BYTES < 4 ? 1 : BYTES / 4];
};

// Rows of tens of thousands of entries pass through L2 once: they are read and written with the
// evict-first policy, which leaves the tokens' own rows (read topk times) there (sort 34 against 41 us,
// unsort 28 against 33, its gradients 57 against 61).
template <int BYTES>
__device__ __forceinline__ Words<BYTES> load_stream(const void* base, int64_t index) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(base) + index * BYTES;
  Words<BYTES> r;
  if constexpr (BYTES == 2) {
    r.w[0] = __ldcs(reinterpret_cast<const unsigned short*>(p));
  } else if constexpr (BYTES == 4) {
    r.w[0] = __ldcs(reinterpret_cast<const unsigned int*>(p));
  } else if constexpr (BYTES == 8) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
      r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
  }
  return r;
}

template <int BYTES>
__device__ __forceinline__ Words<BYTES> load_words(const void* base, int64_t index) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(base) + index * BYTES;
  Words<BYTES> r;
  if constexpr (BYTES == 2) {
    r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else if constexpr (BYTES == 4) {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (BYTES == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
  }
  return r;
}

template <int BYTES>
__device__ __forceinline__ void store_stream(void* base, int64_t index, const Words<BYTES>& r) {
  uint8_t* p = reinterpret_cast<uint8_t*>(base) + index * BYTES;
  if constexpr (BYTES == 2) {
    __stcs(reinterpret_cast<unsigned short*>(p), (unsigned short)r.w[0]);
  } else if constexpr (BYTES == 4) {
    __stcs(reinterpret_cast<unsigned int*>(p), r.w[0]);
  } else if constexpr (BYTES == 8) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(r.w[0], r.w[1]));
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i)
      __stcs(reinterpret_cast<uint4*>(p) + i, make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]));
  }
}

template <int DT>
struct Elem {
  static constexpr int kBytes = DT == SP24_F32 ? 4 : 2;
  // element k of a vector's words
  template <int BYTES>
  static __device__ __forceinline__ float get(const Words<BYTES>& v, int k) {
    if (DT == SP24_F32) return __uint_as_float(v.w[k]);
    const uint32_t word = v.w[k / 2];
    if (DT == SP24_BF16) return __uint_as_float(k & 1 ? word & 0xffff0000u : word << 16);
    return __half2float(__ushort_as_half((unsigned short)(k & 1 ? word >> 16 : word & 0xffffu)));
  }
  static __device__ __forceinline__ uint32_t bits(float v) {
    if (DT == SP24_F32) return __float_as_uint(v);
    return DT == SP24_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
  }
  template <int V>
  static __device__ __forceinline__ Words<V * kBytes> put(const float (&f)[V]) {
    Words<V * kBytes> r;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (DT == SP24_F32)
        r.w[k] = bits(f[k]);
      else if (k % 2 == 0)
        r.w[k / 2] = bits(f[k]);
      else
        r.w[k / 2] |= bits(f[k]) << 16;
    }
    return r;
  }
};

// ------------------------------------------------------------------ sort
//
// The row of entry i is the number of entries before it in the order (expert, entry number).
//
// Few entries: one warp per entry counts over all of them and moves the entry's row of x, in one
// launch.  Many: three.  The entries are cut into chunks of about sqrt(n); the first launch counts
// each chunk's entries per expert, the second turns an expert's counts into those of earlier chunks
// (one warp per expert) and its last CTA to finish adds up the experts' offsets, the third adds to
// both the equal entries before entry i in its own chunk, and moves the rows.  At 2000 entries over 512
// experts the first takes 7.0 us and the second 7.9, at 4000 14 and 7.9: the border is at 2048.  The
// tables of 40960 entries take 11 us by themselves, most of it three launches; the last one's
// reading of keys overlaps the others' end (14 us without).

struct SortTables {
  const int32_t* routing;
  int64_t n, E;
  int32_t *pos, *src, *row_expert, *offsets;
  const int32_t* before;  // [E + 1][chunks]: entries of expert e (E: the empty slots) in earlier chunks
  const int32_t* first;   // [E + 1]: entries of lower experts
  int64_t chunks;
  int chunk_log;
};

// The expert of an entry; empty slots come after every expert.
__device__ __forceinline__ int entry_key(int32_t id, int64_t E) { return id < 0 || id >= E ? (int)E : id; }

__device__ __forceinline__ void put_entry(const SortTables& t, int64_t i, int key, int row) {
  const bool held = key < t.E;
  t.pos[i] = held ? row : -1;
  t.src[row] = held ? (int32_t)i : -1;
  t.row_expert[row] = held ? key : -1;
}

// A warp copies a row of `vecs` vectors, 8 (then 4) loads in flight per lane.
template <int BYTES, int BATCH>
__device__ __forceinline__ void copy_batches(uint8_t* __restrict__ to, const uint8_t* __restrict__ from, int64_t vecs,
                                             int64_t& c) {
  for (; c + 32 * (BATCH - 1) < vecs; c += 32 * BATCH) {
    Words<BYTES> v[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) v[k] = load_words<BYTES>(from, c + 32 * k);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) store_stream<BYTES>(to, c + 32 * k, v[k]);
  }
}
template <int BYTES>
__device__ __forceinline__ void copy_row(uint8_t* __restrict__ to, const uint8_t* __restrict__ from, int64_t vecs) {
  int64_t c = threadIdx.x & 31;
  copy_batches<BYTES, 8>(to, from, vecs, c);
  copy_batches<BYTES, 4>(to, from, vecs, c);
  copy_batches<BYTES, 1>(to, from, vecs, c);
}

// One warp per entry, then one per offset.
template <int BYTES>
__global__ void __launch_bounds__(32 * kWarps) sort_few_kernel(const __grid_constant__ SortTables t,
                                                               const uint8_t* __restrict__ x, int topk,
                                                               int64_t row_bytes, uint8_t* __restrict__ xs) {
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * kWarps + (threadIdx.x >> 5), n = (int)t.n;
  begin();
  if (i >= n + t.E + 1) return;
  const int32_t id = i < n ? t.routing[i] : i - n;
  const int key = entry_key(id, t.E);
  int before = 0;  // i >= n: all entries of lower experts
  for (int j = lane; j < n; j += 32) {
    const int k = entry_key(t.routing[j], t.E);
    before += k < key || (k == key && j < i && i < n);
  }
  before = __reduce_add_sync(kFull, before);
  if (i >= n) {
    if (lane == 0) t.offsets[i - n] = before;
    return;
  }
  if (lane == 0) {
    if (key == t.E && id != -1) set_dev_error(SP24_ERR_INVALID_ARG);
    put_entry(t, i, key, before);
  }
  if (key == t.E || !x) return;
  copy_row<BYTES>(xs + (int64_t)before * row_bytes, x + (i / topk) * row_bytes, row_bytes / BYTES);
}

// Each CTA counts one chunk, kCounters experts at a time.
__global__ void __launch_bounds__(256) sort_count_kernel(const int32_t* __restrict__ routing, int64_t n, int64_t E,
                                                         int chunk_log, int64_t chunks, int32_t* __restrict__ counts,
                                                         int32_t* __restrict__ done) {
  extern __shared__ int32_t held[];
  begin();
  if (blockIdx.x == 0 && threadIdx.x == 0) *done = 0;
  const int64_t from = (int64_t)blockIdx.x << chunk_log, to = min(n, from + ((int64_t)1 << chunk_log));
  for (int e0 = 0; e0 <= E; e0 += kCounters) {
    const int span = (int)min((int64_t)kCounters, E + 1 - e0);
    for (int e = threadIdx.x; e < span; e += 256) held[e] = 0;
    __syncthreads();
    for (int64_t j = from + threadIdx.x; j < to; j += 256) {
      const int key = entry_key(routing[j], E) - e0;
      if (key >= 0 && key < span) atomicAdd(&held[key], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < span; e += 256) counts[(int64_t)(e0 + e) * chunks + blockIdx.x] = held[e];
    __syncthreads();
  }
}

constexpr int kScan = 8;  // counts in flight per lane

__device__ __forceinline__ int warp_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(kFull, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// One warp per expert: its counts become those of earlier chunks.  The CTA that finishes last (a
// counter tells; nobody waits) turns the totals into `first` and the offsets.
__global__ void __launch_bounds__(32 * kWarps) sort_scan_kernel(int32_t* __restrict__ counts, int64_t E, int64_t chunks,
                                                                int32_t* __restrict__ first,
                                                                int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ done) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t e = (int64_t)blockIdx.x * kWarps + warp;
  begin();
  if (e <= E) {
    int32_t* const mine = counts + e * chunks;
    int carry = 0;
    for (int64_t c0 = 0; c0 < chunks; c0 += 32 * kScan) {
      int v[kScan];
#pragma unroll
      for (int k = 0; k < kScan; ++k) v[k] = c0 + 32 * k + lane < chunks ? mine[c0 + 32 * k + lane] : 0;
#pragma unroll
      for (int k = 0; k < kScan; ++k) {
        const int upto = warp_scan(v[k]);
        if (c0 + 32 * k + lane < chunks) mine[c0 + 32 * k + lane] = carry + upto - v[k];
        carry += __shfl_sync(kFull, upto, 31);
      }
    }
    if (lane == 0) first[e] = carry;
  }
  __shared__ int last;
  __shared__ int sums[kWarps];
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(done, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  int carry = 0;
  for (int64_t e0 = 0; e0 <= E; e0 += 32 * kWarps) {
    const int64_t at = e0 + threadIdx.x;
    const int v = at <= E ? __ldcg(first + at) : 0;
    const int upto = warp_scan(v);
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int base = carry;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) base += sums[w];
      carry += sums[w];
    }
    if (at <= E) first[at] = offsets[at] = base + upto - v;
    __syncthreads();
  }
}

// kEntries entries per CTA, kParts threads each for the place within the chunk, then one warp per row
// (64 entries of 4 threads: 44 against 41 us, too few rows under way at once).
constexpr int kEntries = 32;
constexpr int kParts = 8;
constexpr int kMaxChunkLog = 11;
template <int BYTES>
__global__ void __launch_bounds__(kParts * kEntries) sort_many_kernel(const __grid_constant__ SortTables t,
                                                                 const uint8_t* __restrict__ x, int topk,
                                                                 int64_t row_bytes, uint8_t* __restrict__ xs) {
  __shared__ int32_t keys[1 << kMaxChunkLog];  // from the chunk's first entry to this CTA's last
  __shared__ int rows[kEntries];
  const int64_t i0 = (int64_t)blockIdx.x * kEntries, from = i0 >> t.chunk_log << t.chunk_log;
  const int mine = (int)min((int64_t)kEntries, t.n - i0), ahead = (int)(i0 - from);
  // the keys are read before the wait: the kernel before this one, the scan, does not write them
  for (int j = threadIdx.x; j < ahead + mine; j += kParts * kEntries) {
    const int32_t id = t.routing[from + j];
    const int key = entry_key(id, t.E);
    if (key == t.E && id != -1 && j >= ahead) set_dev_error(SP24_ERR_INVALID_ARG);
    keys[j] = key;
  }
  __syncthreads();
  const int i = threadIdx.x / kParts, part = threadIdx.x % kParts;
  const int key = i < mine ? keys[ahead + i] : 0;
  int equal = 0;
  if (i < mine)
    for (int j = part; j < ahead + i; j += kParts) equal += keys[j] == key;
#pragma unroll
  for (int d = 1; d < kParts; d <<= 1) equal += __shfl_xor_sync(kFull, equal, d);
  begin();
  if (i < mine && part == 0) {
    const int row = t.first[key] + t.before[key * t.chunks + (i0 >> t.chunk_log)] + equal;
    put_entry(t, i0 + i, key, row);
    rows[i] = key < t.E ? row : -1;
  }
  if (!x) return;
  __syncthreads();
  for (int e = threadIdx.x >> 5; e < mine; e += kParts * kEntries / 32)
    if (rows[e] >= 0)
      copy_row<BYTES>(xs + (int64_t)rows[e] * row_bytes, x + (i0 + e) / topk * row_bytes, row_bytes / BYTES);
}

// Above this many entries the counts are made by chunk: see above.
constexpr int64_t kFew = 2048;

struct SortWs {
  int chunk_log;
  int64_t chunks, first_at, before_at, bytes;
};

SortWs sort_layout(int64_t n, int64_t E) {
  SortWs w{};
  if (n <= kFew) return w;
  w.chunk_log = 8;
  while (w.chunk_log < kMaxChunkLog && ((int64_t)1 << (2 * w.chunk_log)) < n) ++w.chunk_log;
  w.chunks = (n + ((int64_t)1 << w.chunk_log) - 1) >> w.chunk_log;
  w.first_at = 16;
  w.before_at = w.first_at + ((E + 1) * 4 + 15) / 16 * 16;
  w.bytes = w.before_at + (E + 1) * w.chunks * 4;
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

// One warp per 32 W vectors of V columns of one token; the slots in order, kSlots of them in flight:
// five of one vector, but two of two where a token has no more slots (16384 x 2 rows of [2048]: 31
// against 51 us), and two of eight columns where rows allow vectors of one or two (V = 2: 34 against 39
// us at 4096 x 10; V = 1, an odd width of a 16-bit type, takes 104 us either way).
template <int YS, int Y, int V, int W, int kSlots>
__global__ void __launch_bounds__(32 * kWarps) unsort_kernel(const void* __restrict__ ys,
                                                             const int32_t* __restrict__ pos,
                                                             const float* __restrict__ router_w, uint32_t units,
                                                             uint32_t per_row, int topk, int64_t rows, int64_t HV,
                                                             void* __restrict__ y) {
  constexpr int kIn = V * Elem<YS>::kBytes, kOut = V * Elem<Y>::kBytes;
  const int lane = threadIdx.x & 31;
  const uint32_t u = blockIdx.x * kWarps + (threadIdx.x >> 5);
  begin();
  if (u >= units) return;
  const uint32_t t = u / per_row;
  const int64_t c = (int64_t)(u - t * per_row) * (32 * W) + lane;
  const int32_t* const my_pos = pos + (int64_t)t * topk;
  const float* const my_w = router_w + (int64_t)t * topk;
  float acc[W][V];
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int k = 0; k < V; ++k) acc[j][k] = 0.0f;
  for (int s0 = 0; s0 < topk; s0 += kSlots) {
    int r[kSlots];
    float w[kSlots];
    Words<kIn> v[kSlots][W];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const bool slot = s0 + s < topk;
      r[s] = slot ? my_pos[s0 + s] : -1;
      w[s] = slot && router_w ? my_w[s0 + s] : 1.0f;
    }
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const bool held = r[s] >= 0 && r[s] < rows;
      if (!held && r[s] != -1) set_dev_error(SP24_ERR_INVALID_ARG);
      w[s] = held ? w[s] : 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        v[s][j] = Words<kIn>{};
        if (held && c + 32 * j < HV) v[s][j] = load_stream<kIn>(ys, r[s] * HV + c + 32 * j);
      }
    }
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k) acc[j][k] = fmaf(w[s], Elem<YS>::get(v[s][j], k), acc[j][k]);
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
    if (c + 32 * j < HV) store_stream<kOut>(y, (int64_t)t * HV + c + 32 * j, Elem<Y>::put(acc[j]));
}

// One warp per entry: its row of dys, and (DOT) the dot product that is its weight's gradient; kPairs
// loads of either row in flight per lane.
constexpr int kPairs = 4;
template <int YS, int Y, int V, bool DOT>
__global__ void __launch_bounds__(32 * kWarps) unsort_backward_kernel(
    const void* __restrict__ dy, const void* __restrict__ ys, const int32_t* __restrict__ pos,
    const float* __restrict__ router_w, int64_t n, int topk, int64_t rows, int64_t HV, void* __restrict__ dys,
    float* __restrict__ d_router_w) {
  constexpr int kIn = V * Elem<YS>::kBytes, kOut = V * Elem<Y>::kBytes;
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  begin();
  if (i >= n) return;
  const int r = entry_row(pos, i, rows);
  if (r < 0) {
    if (DOT && lane == 0) d_router_w[i] = 0.0f;
    return;
  }
  const float w = router_w ? router_w[i] : 1.0f;
  const int64_t from = (int64_t)((uint32_t)i / (uint32_t)topk) * HV, at = r * HV;
  float dot = 0.0f;
  auto step = [&](int64_t c, const Words<kOut>& g, const Words<kIn>& v) {
    float d[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float a = Elem<Y>::get(g, k);
      if (DOT) dot = fmaf(a, Elem<YS>::get(v, k), dot);
      d[k] = w * a;
    }
    store_stream<kIn>(dys, at + c, Elem<YS>::put(d));
  };
  int64_t c = lane;
  for (; c + 32 * (kPairs - 1) < HV; c += 32 * kPairs) {
    Words<kOut> g[kPairs];
    Words<kIn> v[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      g[j] = load_words<kOut>(dy, from + c + 32 * j);
      v[j] = Words<kIn>{};
      if (DOT) v[j] = load_stream<kIn>(ys, at + c + 32 * j);
    }
#pragma unroll
    for (int j = 0; j < kPairs; ++j) step(c + 32 * j, g[j], v[j]);
  }
  for (; c < HV; c += 32) {
    Words<kIn> v{};
    if (DOT) v = load_stream<kIn>(ys, at + c);
    step(c, load_words<kOut>(dy, from + c), v);
  }
  if (DOT) {
#pragma unroll
    for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(kFull, dot, d);
    if (lane == 0) d_router_w[i] = dot;
  }
}

// Calls f with a tag of the pair of types (one that the header names).
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
  if (E > (1 << 16) || T > INT32_MAX || T * topk > INT32_MAX) return SP24_ERR_UNSUPPORTED;
  *bytes = sort_layout(T * topk, E).bytes;
  return SP24_OK;
}

extern "C" int sp24_moe_sort(const void* x, int dtype, const int32_t* routing, int64_t T, int topk, int64_t E,
                             int64_t H, void* xs, int32_t* pos, int32_t* src, int32_t* row_expert, int32_t* offsets,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  const int eb = elem_bytes(dtype);
  if (!eb) return SP24_ERR_DTYPE;
  if (T < 0 || topk < 1 || E < 1 || H < 0) return SP24_ERR_SHAPE;
  if (E > (1 << 16) || T > INT32_MAX || T * topk > INT32_MAX) return SP24_ERR_UNSUPPORTED;
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
  int st = SP24_OK;
  if (ws.bytes) {
    uint8_t* const base = reinterpret_cast<uint8_t*>(workspace);
    int32_t* const done = reinterpret_cast<int32_t*>(base);
    int32_t* const first = reinterpret_cast<int32_t*>(base + ws.first_at);
    int32_t* const before = reinterpret_cast<int32_t*>(base + ws.before_at);
    const int64_t counters = E + 1 < kCounters ? E + 1 : kCounters;
    st = launch_after(sort_count_kernel, (unsigned)ws.chunks, 256, (size_t)counters * 4, s, routing, n, E, ws.chunk_log,
                      ws.chunks, before, done);
    if (st) return st;
    st = launch_after(sort_scan_kernel, (unsigned)((E + kWarps) / kWarps), 32 * kWarps, 0, s, before, E, ws.chunks, first,
                      offsets, done);
    if (st) return st;
    t.first = first;
    t.before = before;
  }
  const int64_t row = H * eb;
  const uint8_t* from = H ? reinterpret_cast<const uint8_t*>(x) : nullptr;
  uint8_t* to = reinterpret_cast<uint8_t*>(xs);
  auto run = [&](auto bytes) {
    constexpr int B = decltype(bytes)::value;
    if (ws.bytes)
      return launch_after(sort_many_kernel<B>, (unsigned)((n + kEntries - 1) / kEntries), kParts * kEntries, 0, s, t,
                          from, topk, row, to);
    return launch_after(sort_few_kernel<B>, (unsigned)((n + E + kWarps) / kWarps), 32 * kWarps, 0, s, t, from, topk, row,
                        to);
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
      auto go = [&](auto wide, auto slots) {
        constexpr int W = decltype(wide)::value, S = decltype(slots)::value;
        const int64_t per_row = (H / V + 32 * W - 1) / (32 * W), units = T * per_row;
        if (units > INT32_MAX) return (int)SP24_ERR_UNSUPPORTED;  // more than any device's memory holds
        return launch_after(unsort_kernel<decltype(p)::ys, decltype(p)::y, V, W, S>,
                            (unsigned)((units + kWarps - 1) / kWarps), 32 * kWarps, 0, s, ys, pos, router_w,
                            (uint32_t)units, (uint32_t)per_row, topk, rows, H / V, y);
      };
      constexpr int W = V >= 4 ? 2 : 8 / V;
      if (topk <= 2) return go(std::integral_constant<int, W>{}, std::integral_constant<int, 2>{});
      if (V <= 2) return go(std::integral_constant<int, W>{}, std::integral_constant<int, 2>{});
      return go(std::integral_constant<int, 1>{}, std::integral_constant<int, 5>{});
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
      const unsigned ctas = (unsigned)((n + kWarps - 1) / kWarps);
      if (d_router_w)
        return launch_after(unsort_backward_kernel<decltype(p)::ys, decltype(p)::y, V, true>, ctas, 32 * kWarps, 0, s, dy, ys,
                            pos, router_w, n, topk, rows, H / V, dys, d_router_w);
      return launch_after(unsort_backward_kernel<decltype(p)::ys, decltype(p)::y, V, false>, ctas, 32 * kWarps, 0, s, dy, ys,
                          pos, router_w, n, topk, rows, H / V, dys, nullptr);
    };
    if (v == 8) return run(std::integral_constant<int, 8>{});
    if (v == 4) return run(std::integral_constant<int, 4>{});
    return v == 2 ? run(std::integral_constant<int, 2>{}) : run(std::integral_constant<int, 1>{});
  });
}
