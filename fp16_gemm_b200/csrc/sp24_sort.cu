// Token sort and unsort of the routed feed-forward: rows of x into expert order, expert outputs
// back in token order with the router weights applied, and the gradients of both (definitions in
// sp24.h; [P1] "Concurrency, not sparsity, is the lever" names the routed model).
//
// Everything here moves rows; nothing is multiplied more than once, so HBM is the bound.  Measured at
// 4096 tokens x 10 slots, rows of 2048 bf16 entries (185 MB moved one way, 28 us at the copy rate): sort 41 us
// (10.6 of them its tables), its gradient 28 us, unsort 28 us, its gradients 56 us (354 MB, 54 us).  A decode
// step (8 tokens): 2.4 to 3.9 us each, the time of a launch and two or three dependent loads.
//
// Figures are the GPU's time for a call, in a replayed graph of calls on tensors that take turns.  "a
// against b" is what both forms took side by side when the choice between them was made, a the one that is here.
#include "sp24_launch.cuh"

namespace sp24 {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kMaxUnsortTopk = 64;
constexpr int kCounters = 8192;  // counters of one pass over a chunk (32 KB of shared memory)
constexpr int kMaxChunkLog = 11;

// ------------------------------------------------------------------ element access

// BYTES (4 to 32) consecutive bytes as 32-bit words, moved with accesses of at most 16 bytes.
template <int BYTES>
struct Words {
  uint32_t w[BYTES / 4];
};

// Rows of tens of thousands of entries pass through L2 once: they are read and written with the
// evict-first policy (STREAM), which leaves the tokens' own rows (read topk times) there (4096 x 10 rows of
// [2048]: sort 41 against 42 us, its gradient 28 against 32, unsort 28 against 32; its gradients lose by it,
// 55.6 against 54.8).
template <bool STREAM, typename T>
__device__ __forceinline__ T load_as(const uint8_t* p) {
  return STREAM ? __ldcs(reinterpret_cast<const T*>(p)) : *reinterpret_cast<const T*>(p);
}
template <bool STREAM, int BYTES>
__device__ __forceinline__ void load_vec(uint32_t* w, const uint8_t* p) {
  if constexpr (BYTES == 4) {
    w[0] = load_as<STREAM, unsigned int>(p);
  } else if constexpr (BYTES == 8) {
    const uint2 v = load_as<STREAM, uint2>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 v = load_as<STREAM, uint4>(p + 16 * i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}
template <int BYTES>
__device__ __forceinline__ void store_vec(uint8_t* p, const Words<BYTES>& r) {
  if constexpr (BYTES == 4) {
    __stcs(reinterpret_cast<unsigned int*>(p), r.w[0]);
  } else if constexpr (BYTES == 8) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(r.w[0], r.w[1]));
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i)
      __stcs(reinterpret_cast<uint4*>(p) + i, make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]));
  }
}

// Rows of whole words (4, 8, 16 bytes) are moved by those.  Rows of 16-bit elements that start between
// words ("ragged": odd widths, odd bases) are stored with aligned 16-byte vectors all the same, what is
// ahead of the first and behind the last one by elements.  What a vector is made of is read as the
// aligned 16-byte pieces around it and shifted, by the same amount all along a row.  4096 x 10 rows of
// 2047 bf16 entries, against 2-byte accesses: sort 46 against 56 us, unsort 55 against 103, its
// gradients 84 against 110 (58, 57 and 91 us on tensors that take turns).  What is left are the shifts'
// instructions; where words do, they are faster (2046 entries: 51, 36 and 77 us).
template <int BYTES, bool RAGGED>
struct Window {
  uint32_t w[BYTES / 4 + (RAGGED ? 4 : 0)];
};

// A row read by vectors of BYTES bytes, the first of which starts at p.
template <int BYTES, bool RAGGED, bool STREAM>
struct RowReader {
  const uint8_t* at;
  int shift;  // ragged: bytes between the aligned piece and the vector
  __device__ __forceinline__ void start(const uint8_t* p) {
    shift = RAGGED ? (int)((uintptr_t)p & 15) : 0;
    at = p - shift;
  }
  // Whether the pieces of vectors c0 to c1 - 1 start at or after lo, and end at or before hi.
  __device__ __forceinline__ bool after(const uint8_t* lo, int64_t c0) const { return at + c0 * BYTES >= lo; }
  __device__ __forceinline__ bool before(const uint8_t* hi, int64_t c1) const {
    return at + c1 * BYTES + (shift ? 16 : 0) <= hi;
  }
  // Starts the loads of vector c.
  __device__ __forceinline__ Window<BYTES, RAGGED> open(int64_t c, bool want) const {
    Window<BYTES, RAGGED> r{};
    const uint8_t* const p = at + c * BYTES;
    if (want) load_vec<STREAM, BYTES>(r.w, p);
    if constexpr (RAGGED)
      if (want && shift) load_vec<STREAM, 16>(r.w + BYTES / 4, p + BYTES);
    return r;
  }
  // The vector out of its pieces.
  __device__ __forceinline__ Words<BYTES> take(Window<BYTES, RAGGED>& v) const {
    Words<BYTES> r;
    if constexpr (RAGGED) {
      const bool two = shift & 8, one = shift & 4;
#pragma unroll
      for (int i = 0; i < BYTES / 4 + 2; ++i) v.w[i] = two ? v.w[i + 2] : v.w[i];
#pragma unroll
      for (int i = 0; i < BYTES / 4 + 1; ++i) v.w[i] = one ? v.w[i + 1] : v.w[i];
#pragma unroll
      for (int i = 0; i < BYTES / 4; ++i) r.w[i] = __funnelshift_r(v.w[i], v.w[i + 1], 8 * (shift & 2));
    } else {
#pragma unroll
      for (int i = 0; i < BYTES / 4; ++i) r.w[i] = v.w[i];
    }
    return r;
  }
};

// A row of len elements, `pad` of which fit ahead of it in its first 16 bytes, as vectors c0 to c1 - 1
// of V (vector c from element c V - pad) and as single elements: the first `head` and those from
// `tail` on, at most 2 V - 1 of either.
struct Split {
  int c0, c1, head, tail, edges;
  template <int V>
  __device__ __forceinline__ void make(int len, int pad) {
    c0 = pad ? 1 : 0, c1 = (len + pad) / V;
  }
  // Vectors whose pieces the tensor [lo, hi) does not hold whole are left to the single elements.
  template <typename Reader>
  __device__ __forceinline__ void clip(const Reader& in, const uint8_t* lo, const uint8_t* hi) {
    if (!in.after(lo, c0)) ++c0;
    if (!in.before(hi, c1)) --c1;
  }
  template <int V>
  __device__ __forceinline__ void close(int len, int pad) {
    head = min(len, c0 * V - pad);
    tail = max(head, c1 * V - pad);
    edges = head + len - tail;
  }
  __device__ __forceinline__ int column(int edge) const { return edge < head ? edge : tail + edge - head; }
};

// Elements of a row ahead of its first that its 16-byte piece holds.
template <int EB, bool RAGGED>
__device__ __forceinline__ int row_pad(const uint8_t* row) {
  return RAGGED ? (int)((uintptr_t)row & 15) / EB : 0;
}
// Vectors of V that hold any row of len elements.
__host__ __device__ __forceinline__ int row_vecs(int64_t len, int V, bool ragged) {
  return (int)(ragged ? (len + 2 * V - 2) / V : len / V);
}

// Lanes that share a row of `vecs` vectors, as a power of two: four vectors each, or all lanes.  With a
// warp for every row, the gradients of 16384 x 10 rows of 16, 64 and 256 bf16 entries took 47, 50 and
// 71 us, so 5, 10 and 33.
int row_lanes_log(int64_t vecs, bool ragged) {
  int log = ragged ? 3 : 0;  // the elements at a row's ends have lanes too
  while (log < 5 && ((int64_t)4 << log) < vecs) ++log;
  return log;
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
  static __device__ __forceinline__ float at(const uint8_t* row, int i) {
    if (DT == SP24_F32) return reinterpret_cast<const float*>(row)[i];
    const uint32_t v = reinterpret_cast<const uint16_t*>(row)[i];
    return DT == SP24_BF16 ? __uint_as_float(v << 16) : __half2float(__ushort_as_half((unsigned short)v));
  }
  static __device__ __forceinline__ void set(uint8_t* row, int i, float v) {
    if (DT == SP24_F32)
      reinterpret_cast<float*>(row)[i] = v;
    else
      reinterpret_cast<uint16_t*>(row)[i] = (uint16_t)bits(v);
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
        r.w[k] = __float_as_uint(f[k]);
      else if (k % 2 == 0)
        r.w[k / 2] = DT == SP24_BF16 ? pair_bits(__floats2bfloat162_rn(f[k], f[k + 1]))
                                     : pair_bits(__floats2half2_rn(f[k], f[k + 1]));
    }
    return r;
  }
  template <typename P>
  static __device__ __forceinline__ uint32_t pair_bits(P p) {
    return *reinterpret_cast<uint32_t*>(&p);
  }
};

// ------------------------------------------------------------------ sort
//
// The row of entry i is the number of entries before it in the order (expert, entry number).
//
// Few entries: one warp per entry counts over all of them and moves the entry's row of x, in one
// launch.  Many: four.  The entries are cut into chunks of about sqrt(n); the first launch counts
// each chunk's entries per expert, the second turns an expert's counts into those of earlier chunks
// (one warp per expert) and its last CTA to finish adds up the experts' offsets, the third adds to
// both the equal entries before entry i in its own chunk, the fourth moves the rows.  At 2000 entries over
// 512 experts the first way takes 7.0 us and the second 8.2, at 4000 14 and 8.3: the border is at 2048.  The
// tables take 10.6 us at 40960 entries and 13.4 at 163840, most of it launches and dependent loads.

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

// `lanes` lanes copy a row of `vecs` vectors, 8 (then 4) loads in flight per lane.
template <int BYTES, int BATCH>
__device__ __forceinline__ void copy_batches(uint8_t* to, const uint8_t* from, int vecs,
                                             int lanes, int& c) {
  for (; c + lanes * (BATCH - 1) < vecs; c += lanes * BATCH) {
    Words<BYTES> v[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) load_vec<false, BYTES>(v[k].w, from + (int64_t)(c + lanes * k) * BYTES);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) store_vec(to + (int64_t)(c + lanes * k) * BYTES, v[k]);
  }
}
template <int BYTES>
__device__ __forceinline__ void copy_words(uint8_t* to, const uint8_t* from, int64_t bytes,
                                           int lanes, int sub) {
  int c = sub;
  const int vecs = (int)(bytes / BYTES);
  copy_batches<BYTES, 8>(to, from, vecs, lanes, c);
  copy_batches<BYTES, 4>(to, from, vecs, lanes, c);
  Words<BYTES> v[3];
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (c + lanes * k < vecs) load_vec<false, BYTES>(v[k].w, from + (int64_t)(c + lanes * k) * BYTES);
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (c + lanes * k < vecs) store_vec(to + (int64_t)(c + lanes * k) * BYTES, v[k]);
}
__device__ __forceinline__ void copy_ragged(uint8_t* to, const uint8_t* from, int64_t bytes,
                                            const uint8_t* lo, const uint8_t* hi, int lanes, int sub) {
  constexpr int kBatch = 4;
  const int len = (int)(bytes / 2), pad = row_pad<2, true>(to);
  RowReader<16, true, false> in;
  in.start(from - 2 * pad);
  Split part;
  part.make<8>(len, pad);
  part.clip(in, lo, hi);
  part.close<8>(len, pad);
  uint16_t edge = 0;  // read ahead of the vectors, written after them
  if (sub < part.edges) edge = reinterpret_cast<const uint16_t*>(from)[part.column(sub)];
  for (int c = part.c0 + sub; c < part.c1; c += kBatch * lanes) {
    Window<16, true> v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) v[k] = in.open(c + k * lanes, c + k * lanes < part.c1);
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (c + k * lanes < part.c1) store_vec(to - 2 * pad + (int64_t)(c + k * lanes) * 16, in.take(v[k]));
  }
  for (int e = sub; e < part.edges; e += lanes)
    reinterpret_cast<uint16_t*>(to)[part.column(e)] =
        e == sub ? edge : reinterpret_cast<const uint16_t*>(from)[part.column(e)];
}
// BYTES: 16, 8, 4, or 2 for ragged rows.  FULL: all lanes of a warp (known strides: sort 40.5 against 41.3
// us, of 16384 x 8 rows of [512] fp32 66 against 71).
template <int BYTES, bool FULL>
__device__ __forceinline__ void copy_row(uint8_t* to, const uint8_t* from, int64_t bytes,
                                         const uint8_t* lo, const uint8_t* hi, int lanes_log) {
  const int lanes = FULL ? 32 : 1 << lanes_log, sub = threadIdx.x & (lanes - 1);
  if constexpr (BYTES == 2)
    copy_ragged(to, from, bytes, lo, hi, lanes, sub);
  else
    copy_words<BYTES>(to, from, bytes, lanes, sub);
}

// One warp per entry, then one per offset.
template <int BYTES>
__global__ void __launch_bounds__(32 * kWarps) sort_few_kernel(const __grid_constant__ SortTables t,
                                                               const uint8_t* x, int topk,
                                                               int64_t row_bytes, uint8_t* xs) {
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
  copy_row<BYTES, true>(xs + (int64_t)before * row_bytes, x + (i / topk) * row_bytes, row_bytes, x,
                   x + n / topk * row_bytes, 5);
}

// Each CTA counts one chunk, kCounters experts at a time.
__global__ void __launch_bounds__(256) sort_count_kernel(const int32_t* routing, int64_t n, int64_t E,
                                                         int chunk_log, int64_t chunks, int32_t* counts,
                                                         int32_t* done) {
  extern __shared__ int32_t held[];
  begin();
  if (blockIdx.x == 0 && threadIdx.x == 0) *done = 0;
  constexpr int kEach = (1 << kMaxChunkLog) / 256;
  const int64_t from = (int64_t)blockIdx.x << chunk_log, to = min(n, from + ((int64_t)1 << chunk_log));
  int key[kEach];  // a thread's entries, all loads in flight together
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int64_t j = from + threadIdx.x + 256 * k;
    key[k] = j < to ? entry_key(routing[j], E) : -1;
  }
  for (int e0 = 0; e0 <= E; e0 += kCounters) {
    const int span = (int)min((int64_t)kCounters, E + 1 - e0);
    for (int e = threadIdx.x; e < span; e += 256) held[e] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (key[k] >= e0 && key[k] - e0 < span) atomicAdd(&held[key[k] - e0], 1);
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
__global__ void __launch_bounds__(32 * kWarps) sort_scan_kernel(int32_t* counts, int64_t E, int64_t chunks,
                                                                int32_t* first,
                                                                int32_t* offsets,
                                                                int32_t* done) {
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

// One CTA per chunk: an entry's row is its expert's first, the expert's entries of earlier chunks, and
// those of this chunk before it: the lanes of its warp with its key by a match, the warps before it by
// counters in shared memory that the warps pass through in turn.  kCounters experts at a time.
// (Comparing every entry with all before it in its chunk: 20 us for the tables of 163840 entries.)
constexpr int kRankWarps = 16;
__global__ void __launch_bounds__(32 * kRankWarps) sort_rank_kernel(const __grid_constant__ SortTables t) {
  extern __shared__ int32_t held[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t from = (int64_t)blockIdx.x << t.chunk_log;
  const int mine = (int)min((int64_t)1 << t.chunk_log, t.n - from);
  begin();
  for (int e0 = 0; e0 <= t.E; e0 += kCounters) {
    const int span = (int)min((int64_t)kCounters, t.E + 1 - e0);
    for (int e = threadIdx.x; e < span; e += 32 * kRankWarps) held[e] = 0;
    __syncthreads();
    for (int r0 = 0; r0 < mine; r0 += 32 * kRankWarps) {
      const int j = r0 + threadIdx.x;
      const int32_t id = j < mine ? t.routing[from + j] : -1;
      const int key = entry_key(id, t.E) - e0;
      const bool in = j < mine && key >= 0 && key < span;
      const unsigned same = __match_any_sync(kFull, in ? key : -1);
      const int leader = __ffs(same) - 1;
      int row = in ? t.first[e0 + key] + t.before[(e0 + key) * t.chunks + blockIdx.x] : 0;
      int base = 0;
      const int warps = min(kRankWarps, (mine - r0 + 31) / 32);
      for (int w = 0; w < warps; ++w) {
        if (w == warp && in && lane == leader) {
          base = held[key];
          held[key] = base + __popc(same);
        }
        __syncthreads();
      }
      base = __shfl_sync(kFull, base, leader);
      if (in) {
        if (e0 + key == t.E && id != -1) set_dev_error(SP24_ERR_INVALID_ARG);
        row += base + __popc(same & ((1u << lane) - 1));
        put_entry(t, from + j, e0 + key, row);
      }
    }
    __syncthreads();
  }
}

// 1 << lanes_log lanes (FULL: a warp) copy an entry's row.
template <int BYTES, bool FULL>
__global__ void __launch_bounds__(32 * kWarps) sort_copy_kernel(const int32_t* pos, int64_t n,
                                                                const uint8_t* x, int topk,
                                                                int64_t row_bytes, uint8_t* xs,
                                                                int lanes_log) {
  if (FULL) lanes_log = 5;
  const int64_t i = ((int64_t)blockIdx.x * (32 * kWarps) + threadIdx.x) >> lanes_log;
  begin();
  const int row = i < n ? pos[i] : -1;
  if (row >= 0)
    copy_row<BYTES, FULL>(xs + (int64_t)row * row_bytes, x + (int64_t)((uint32_t)i / (uint32_t)topk) * row_bytes,
                          row_bytes, x, x + n / topk * row_bytes, lanes_log);
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

// One warp (FULL) per 32 W vectors of V columns of one token, or 1 << lanes_log lanes where a row has no
// more vectors (16384 x 10 rows of [64]: 4 against 11 us); the slots in order, kSlots of them in flight:
// five of one vector, but two of two where a token has no more slots (16384 x 2 rows of [2048]: 31
// against 51 us), and two of eight columns where rows allow vectors of one or two (V = 2: 31 against 39
// us at 4096 x 10).
template <int YS, int Y, int V, bool RAGGED, bool FULL, int W, int kSlots>
__global__ void __launch_bounds__(32 * kWarps, !RAGGED ? 1 : YS == SP24_F32 ? 2 : 3)
    unsort_kernel(const uint8_t* ys, const int32_t* pos, const float* router_w,
                  uint32_t units, uint32_t per_row, int topk, int64_t rows, int64_t H, uint8_t* y,
                  int lanes_log) {
  constexpr int kIn = Elem<YS>::kBytes, kOut = Elem<Y>::kBytes;
  if (FULL) lanes_log = 5;
  const int step = 1 << lanes_log;
  const uint32_t u = (uint32_t)(((int64_t)blockIdx.x * (32 * kWarps) + threadIdx.x) >> lanes_log);
  begin();
  if (u >= units) return;
  const int64_t t = u / per_row;
  const uint8_t* const end = ys + rows * H * kIn;
  uint8_t* const row = y + t * H * kOut;
  const int64_t c = (int64_t)(u - (uint32_t)t * per_row) * (step * W) + (threadIdx.x & (step - 1));
  const int pad = row_pad<kOut, RAGGED>(row), vecs = (int)((H + pad + V - 1) / V);
  const int32_t* const my_pos = pos + t * topk;
  const float* const my_w = router_w + t * topk;
  float acc[W][V];
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int k = 0; k < V; ++k) acc[j][k] = 0.0f;
  for (int s0 = 0; s0 < topk; s0 += kSlots) {
    int r[kSlots];
    float w[kSlots];
    RowReader<V * kIn, RAGGED, true> in[kSlots];
    Window<V * kIn, RAGGED> v[kSlots][W];
    bool inside = true;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const bool slot = s0 + s < topk;
      r[s] = slot ? my_pos[s0 + s] : -1;
      w[s] = slot && router_w ? my_w[s0 + s] : 1.0f;
    }
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      if (r[s] < 0 || r[s] >= rows) {
        if (r[s] != -1) set_dev_error(SP24_ERR_INVALID_ARG);
        r[s] = -1, w[s] = 0.0f;
      }
      in[s].start(ys + (max(r[s], 0) * H - pad) * kIn);
      // a row between others of 48 bytes or more: its pieces are in them
      if (RAGGED && r[s] >= 0 && (r[s] == 0 || r[s] == rows - 1 || H * kIn < 48))
        inside &= in[s].after(ys, c) && in[s].before(end, min((int64_t)vecs, c + (W - 1) * step + 1));
    }
    if (RAGGED && !inside) {  // a vector at an end of ys: by elements
      for (int s = s0; s < min(s0 + kSlots, topk); ++s) {
        const int at = my_pos[s];
        if (at < 0 || at >= rows) continue;
        const float weight = router_w ? my_w[s] : 1.0f;
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const int64_t i = (c + j * step) * V - pad + k;
            if (i >= 0 && i < H) acc[j][k] = fmaf(weight, Elem<YS>::at(ys + at * H * kIn, (int)i), acc[j][k]);
          }
      }
      continue;
    }
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
#pragma unroll
      for (int j = 0; j < W; ++j) v[s][j] = in[s].open(c + j * step, r[s] >= 0 && c + j * step < vecs);
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const Words<V * kIn> a = in[s].take(v[s][j]);
#pragma unroll
        for (int k = 0; k < V; ++k) acc[j][k] = fmaf(w[s], Elem<YS>::get(a, k), acc[j][k]);
      }
  }
#pragma unroll
  for (int j = 0; j < W; ++j) {
    const int64_t i = (c + j * step) * V - pad;
    if (RAGGED ? i >= 0 && i + V <= H : i < H)
      store_vec(row + i * kOut, Elem<Y>::put(acc[j]));
    else if (RAGGED && i < H)
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (i + k >= 0 && i + k < H) Elem<Y>::set(row, (int)i + k, acc[j][k]);
  }
}

// 1 << lanes_log lanes per entry: its row of dys, and (DOT) the dot product that is its weight's
// gradient; kPairs loads of either row in flight per lane.
template <bool RAGGED>
constexpr int kPairs = RAGGED ? 2 : 4;
template <int YS, int Y, int V, bool RAGGED, bool DOT, bool FULL>
__global__ void __launch_bounds__(32 * kWarps, RAGGED ? 3 : 1) unsort_backward_kernel(
    const uint8_t* dy, const uint8_t* ys, const int32_t* pos,
    const float* router_w, int64_t n, int topk, int64_t rows, int64_t H, uint8_t* dys,
    float* d_router_w, int lanes_log) {
  if (FULL) lanes_log = 5;
  constexpr int kIn = Elem<YS>::kBytes, kOut = Elem<Y>::kBytes;
  const int sub = threadIdx.x & ((1 << lanes_log) - 1);
  const int64_t i = ((int64_t)blockIdx.x * (32 * kWarps) + threadIdx.x) >> lanes_log;
  begin();
  const int r = i < n ? entry_row(pos, i, rows) : -1;
  float dot = 0.0f;
  if (r >= 0) {
    const float w = router_w ? router_w[i] : 1.0f;
    const uint8_t* const from = dy + (int64_t)((uint32_t)i / (uint32_t)topk) * H * kOut;
    const uint8_t* const with = ys + r * H * kIn;
    uint8_t* const to = dys + r * H * kIn;
    const int pad = row_pad<kIn, RAGGED>(to);
    RowReader<V * kOut, RAGGED, false> gs;
    RowReader<V * kIn, RAGGED, true> vs;
    gs.start(from - pad * kOut);
    vs.start(DOT ? with - pad * kIn : nullptr);
    Split part;
    part.make<V>((int)H, pad);
    float edge = 0.0f, edge_with = 0.0f;
    if (RAGGED) {
      part.clip(gs, dy, dy + n / topk * H * kOut);
      if (DOT) part.clip(vs, ys, ys + rows * H * kIn);
      part.close<V>((int)H, pad);
      if (sub < part.edges) {  // read ahead of the vectors, used after them
        edge = Elem<Y>::at(from, part.column(sub));
        if (DOT) edge_with = Elem<YS>::at(with, part.column(sub));
      }
    }
    uint8_t* const first = to - pad * kIn;
    auto batch = [&](int c, auto all) {
      constexpr bool ALL = decltype(all)::value;
      Window<V * kOut, RAGGED> g[kPairs<RAGGED>];
      Window<V * kIn, RAGGED> v[kPairs<RAGGED>];
#pragma unroll
      for (int j = 0; j < kPairs<RAGGED>; ++j) {
        const int at = c + (j << lanes_log);
        g[j] = gs.open(at, ALL || at < part.c1);
        if (DOT) v[j] = vs.open(at, ALL || at < part.c1);
      }
#pragma unroll
      for (int j = 0; j < kPairs<RAGGED>; ++j) {
        const int at = c + (j << lanes_log);
        if (!ALL && at >= part.c1) continue;
        const Words<V * kOut> a = gs.take(g[j]);
        Words<V * kIn> b{};
        if (DOT) b = vs.take(v[j]);
        float d[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float gk = Elem<Y>::get(a, k);
          if (DOT) dot = fmaf(gk, Elem<YS>::get(b, k), dot);
          d[k] = w * gk;
        }
        store_vec(first + (int64_t)at * (V * kIn), Elem<YS>::put(d));
      }
    };
    const int stride = kPairs<RAGGED> << lanes_log;
    int c = part.c0 + sub;
    for (; c - sub + stride <= part.c1; c += stride) batch(c, std::true_type{});
    if (c < part.c1) batch(c, std::false_type{});
    if (RAGGED)
      for (int e = sub; e < part.edges; e += 1 << lanes_log) {
        const int col = part.column(e);
        if (e != sub) {
          edge = Elem<Y>::at(from, col);
          if (DOT) edge_with = Elem<YS>::at(with, col);
        }
        if (DOT) dot = fmaf(edge, edge_with, dot);
        Elem<YS>::set(to, col, w * edge);
      }
  }
  if (DOT) {
    for (int d = 1 << lanes_log >> 1; d; d >>= 1) dot += __shfl_xor_sync(kFull, dot, d);
    if (sub == 0 && i < n) d_router_w[i] = dot;
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

// Calls f with the vector and whether rows are ragged (vectors of 8, where a 16-bit type has no two).
template <int YS, int Y, typename F>
int by_vec(int v, F f) {
  if constexpr (YS == SP24_F32 && Y == SP24_F32) {
    if (v == 1) return f(std::integral_constant<int, 1>{}, std::false_type{});
  } else {
    if (v == 8) return f(std::integral_constant<int, 8>{}, std::false_type{});
    if (v == 1) return f(std::integral_constant<int, 8>{}, std::true_type{});
  }
  if (v == 4) return f(std::integral_constant<int, 4>{}, std::false_type{});
  return f(std::integral_constant<int, 2>{}, std::false_type{});
}

int check_unsort(int ys_dtype, int y_dtype, int64_t T, int topk, int64_t rows, int64_t H) {
  if (!elem_bytes(ys_dtype) || !elem_bytes(y_dtype)) return SP24_ERR_DTYPE;
  if (ys_dtype != SP24_F32 && y_dtype != SP24_F32 && ys_dtype != y_dtype) return SP24_ERR_DTYPE;
  if (T < 0 || topk < 1 || rows < 0 || H < 0) return SP24_ERR_SHAPE;
  if (topk > kMaxUnsortTopk || H > (1 << 30) || T > INT32_MAX || rows > INT32_MAX || T * topk > INT32_MAX)
    return SP24_ERR_UNSUPPORTED;
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
  if (E > (1 << 16) || H > (1 << 30) || T > INT32_MAX || T * topk > INT32_MAX) return SP24_ERR_UNSUPPORTED;
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
  if (ws.bytes) {
    const int64_t counters = E + 1 < kCounters ? E + 1 : kCounters;
    st = launch_after(sort_rank_kernel, (unsigned)ws.chunks, 32 * kRankWarps, (size_t)counters * 4, s, t);
    if (st || !from) return st;
  }
  auto run = [&](auto tag) {
    constexpr int B = decltype(tag)::value;
    if (!ws.bytes)
      return launch_after(sort_few_kernel<B>, (unsigned)((n + E + kWarps) / kWarps), 32 * kWarps, 0, s, t, from, topk, row,
                          to);
    const int log = row_lanes_log(row / (B == 2 ? 16 : B), B == 2);
    const unsigned ctas = (unsigned)(((n << log) + 32 * kWarps - 1) / (32 * kWarps));
    if (log == 5)
      return launch_after(sort_copy_kernel<B, true>, ctas, 32 * kWarps, 0, s, pos, n, from, topk, row, to, log);
    return launch_after(sort_copy_kernel<B, false>, ctas, 32 * kWarps, 0, s, pos, n, from, topk, row, to, log);
  };
  if (row % 16 == 0 && aligned(x, 16) && aligned(xs, 16)) return run(std::integral_constant<int, 16>{});
  if (row % 8 == 0 && aligned(x, 8) && aligned(xs, 8)) return run(std::integral_constant<int, 8>{});
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
    constexpr int YS = decltype(p)::ys, Y = decltype(p)::y;
    return by_vec<YS, Y>(v, [&](auto vec, auto ragged) {
      constexpr int V = decltype(vec)::value;
      constexpr bool R = decltype(ragged)::value;
      const int vecs = row_vecs(H, V, R);
      auto go = [&](auto full, auto wide, auto slots, int log) {
        constexpr int W = decltype(wide)::value, S = decltype(slots)::value;
        const int64_t part = (int64_t)W << log, per_row = (vecs + part - 1) / part, units = T * per_row;
        if (units > INT32_MAX) return (int)SP24_ERR_UNSUPPORTED;  // more than any device's memory holds
        return launch_after(unsort_kernel<YS, Y, V, R, decltype(full)::value, W, S>,
                            (unsigned)(((units << log) + 32 * kWarps - 1) / (32 * kWarps)), 32 * kWarps, 0, s,
                            reinterpret_cast<const uint8_t*>(ys), pos, router_w, (uint32_t)units, (uint32_t)per_row,
                            topk, rows, H, reinterpret_cast<uint8_t*>(y), log);
      };
      constexpr std::integral_constant<int, 1> one{};
      constexpr std::integral_constant<int, 2> two{};
      constexpr std::integral_constant<int, 5> five{};
      constexpr std::integral_constant<int, V >= 4 ? 2 : 8 / V> wide{};
      if (vecs <= 16) {
        int log = 0;
        while ((1 << log) < vecs) ++log;
        return go(std::false_type{}, one, five, log);
      }
      if constexpr (V <= 2) return go(std::true_type{}, wide, two, 5);
      if (topk <= 2) return go(std::true_type{}, wide, two, 5);
      return go(std::true_type{}, one, five, 5);
    });
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
  const int v = vec_elems(H, d_router_w ? ys : nullptr, ei, dy, eo, dys, ei);
  cudaStream_t s = as_stream(stream);
  const int64_t n = T * topk;
  return by_pair(ys_dtype, y_dtype, [&](auto p) {
    constexpr int YS = decltype(p)::ys, Y = decltype(p)::y;
    return by_vec<YS, Y>(v, [&](auto vec, auto ragged) {
      constexpr int V = decltype(vec)::value;
      constexpr bool R = decltype(ragged)::value;
      const int log = row_lanes_log(row_vecs(H, V, R), R);
      const int64_t ctas = ((n << log) + 32 * kWarps - 1) / (32 * kWarps);
      auto go = [&](auto dot, auto full) {
        return launch_after(unsort_backward_kernel<YS, Y, V, R, decltype(dot)::value, decltype(full)::value>,
                            (unsigned)ctas, 32 * kWarps, 0, s, reinterpret_cast<const uint8_t*>(dy),
                            reinterpret_cast<const uint8_t*>(ys), pos, router_w, n, topk, rows, H, reinterpret_cast<uint8_t*>(dys), d_router_w, log);
      };
      if (log == 5) return d_router_w ? go(std::true_type{}, std::true_type{}) : go(std::false_type{}, std::true_type{});
      return d_router_w ? go(std::true_type{}, std::false_type{}) : go(std::false_type{}, std::false_type{});
    });
  });
}
