// The kernel of sp24_gemv_w4 / sp24_gemv_w4_grouped; each type of x is a translation unit of its own.
#pragma once

#include <atomic>

#include "sp24_launch.cuh"
#include "sp24_tc.cuh"
#include "sp24_w4.cuh"

namespace sp24 {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kTeams = 4, kMulPerTeam = 4, kMulWarps = kTeams * kMulPerTeam;
constexpr int kChunk = 256;     // entries of K per stage: 128 code bytes of each row
constexpr int kTileBytes = 16 * kChunk / 2;
constexpr int kSmemMax = 232448;  // of one CTA

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src));
}
// The part of the sixteen bytes that lies before `end`, zeros for the rest; `base` is the array's start.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, const uint8_t* end, const uint8_t* base) {
  const int n = src + 16 <= end ? 16 : src < end ? (int)(end - src) : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(n ? src : base), "r"(n));
}
// The barrier gets this thread's arrival when all its copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// A bounded wait of the whole warp.  Each lane measures its own time: where the limit falls next to the
// barrier's completion some find it run out and others not, so they agree, and all give up or none.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(kFull, tc::mbar_wait(bar, parity));
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <int XT>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (XT == SP24_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same on top of zero.
template <int XT>
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (XT == SP24_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// The code q as a 16-bit float without a conversion.  Bits below a float's exponent field, alone, are a
// subnormal number, and the numbers up to twice the smallest normal one are evenly spaced: the four
// bits of a code at the bottom of a 16-bit half are q times the smallest subnormal, those above them 16 q
// times it (bf16: with the last exponent bit among them).  One fma by a power of two, which differs by
// 16 between the two places, makes both (q - z) kUnit exactly, where kUnit is a power of two that
// bf16's largest power of two allows; the sums are divided by it at the end.  So a word takes four
// masks, one shift and four fmas.
template <int XT>
struct Expand;
template <>
struct Expand<SP24_BF16> {
  static constexpr float kUnit = 0x1p-6f;
  static constexpr uint32_t kLow = 0x7f007f00u, kHigh = 0x7d007d00u;  // 2^127 and 2^123 (smallest subnormal: 2^-133)
  // -z kUnit in both halves, for z in 0..15: the bits of z as a float, its exponent moved
  static __device__ __forceinline__ uint32_t zero(uint32_t z) {
    const __nv_bfloat162 v = __float2bfloat162_rn((float)(int)z * -kUnit);
    return reinterpret_cast<const uint32_t&>(v);
  }
  // the same from a byte whose low four bits are z
  static __device__ __forceinline__ uint32_t zero_of(uint32_t byte) {
    return fma2((byte & 15u) * 0x10001u, kLow | 0x80008000u, 0x80008000u);
  }
  static __device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    const __nv_bfloat162 r = __hfma2(reinterpret_cast<const __nv_bfloat162&>(a), reinterpret_cast<const __nv_bfloat162&>(b),
                                     reinterpret_cast<const __nv_bfloat162&>(c));
    return reinterpret_cast<const uint32_t&>(r);
  }
};
template <>
struct Expand<SP24_F16> {
  static constexpr float kUnit = 0x1p-10f;
  static constexpr uint32_t kLow = 0x74007400u, kHigh = 0x64006400u;  // 2^14 and 2^10 (smallest subnormal: 2^-24)
  static __device__ __forceinline__ uint32_t zero(uint32_t z) {
    const __half2 v = __float2half2_rn((float)(int)z * -kUnit);
    return reinterpret_cast<const uint32_t&>(v);
  }
  static __device__ __forceinline__ uint32_t zero_of(uint32_t byte) {
    return fma2((byte & 15u) * 0x10001u, kLow | 0x80008000u, 0x80008000u);
  }
  static __device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 r = __hfma2(reinterpret_cast<const __half2&>(a), reinterpret_cast<const __half2&>(b),
                              reinterpret_cast<const __half2&>(c));
    return reinterpret_cast<const uint32_t&>(r);
  }
};

// The eight codes of a word as four pairs of (q - z) kUnit: entries (0, 4), (1, 5), (2, 6), (3, 7).
template <int XT>
__device__ __forceinline__ void expand8(uint32_t word, uint32_t zero, uint32_t (&out)[4]) {
  using X = Expand<XT>;
  const uint32_t up = word >> 8;
  out[0] = X::fma2(word & 0x000f000fu, X::kLow, zero);
  out[1] = X::fma2(word & 0x00f000f0u, X::kHigh, zero);
  out[2] = X::fma2(up & 0x000f000fu, X::kLow, zero);
  out[3] = X::fma2(up & 0x00f000f0u, X::kHigh, zero);
}

// The token tiles of all experts, in expert order: expert e has ceil(rows of e / STEP) of them.
// Everything here is computed by a whole warp together.
struct TokenTile {
  int64_t e, m0, m1;  // expert, first row, end of the expert's rows
};

// Expert e's rows, [first, end); none past the last expert.
__device__ __forceinline__ void expert_rows(const GemvW4& p, int e, int& first, int& end) {
  first = end = 0;
  if (e < p.E) {
    first = max(0, p.offsets[e]);
    end = max(first, min((int)p.M, p.offsets[e + 1]));
  }
}

// Numbers of tiles.  Offsets that ascend give at most M / STEP and one per expert that has rows, which
// the launch knows (p.tile_bound) and keeps below kManyTiles.  Others may name the same rows again and
// again: sums stop at kManyTiles instead of wrapping, and tiles from the bound on are left out.
constexpr unsigned kManyTiles = 1u << 30;

template <int STEP>
__device__ __forceinline__ unsigned tiles_of(int first, int end) {
  return ((unsigned)(end - first) + STEP - 1) / STEP;
}

// The lanes' sum; each has kManyTiles at most.
__device__ __forceinline__ unsigned sum_tiles(unsigned v) {
  const uint64_t all =
      ((uint64_t)__reduce_add_sync(kFull, v >> 16) << 16) + __reduce_add_sync(kFull, v & 0xffffu);
  return (unsigned)min(all, (uint64_t)kManyTiles);
}

// Inclusive sum over the lanes.
__device__ __forceinline__ unsigned scan_tiles(unsigned v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned o = __shfl_up_sync(kFull, v, d);
    if (lane >= d) v = min(v + o, kManyTiles);
  }
  return v;
}

// The tiles of experts 32 b .. 32 b + 31.
template <int STEP>
__device__ __forceinline__ unsigned block_tiles(const GemvW4& p, int b) {
  int first, end;
  expert_rows(p, 32 * b + (threadIdx.x & 31), first, end);
  return sum_tiles(tiles_of<STEP>(first, end));
}

// A CTA's warps share the counting: `table` holds block_tiles of the first kBlocks blocks.
constexpr int kBlocks = 192;

template <int STEP, typename F>
__device__ __forceinline__ void each_32_blocks(const GemvW4& p, const unsigned* table, F f) {
  const int lane = threadIdx.x & 31, blocks = (int)((p.E + 31) / 32);
  for (int b0 = 0; b0 < blocks; b0 += 32) {
    unsigned mine = b0 + lane < min(blocks, kBlocks) ? table[b0 + lane] : 0;
    for (int b = max(b0, kBlocks); b < min(blocks, b0 + 32); ++b) {  // experts that the table has no room for
      const unsigned s = block_tiles<STEP>(p, b);
      if (b == b0 + lane) mine = s;
    }
    if (f(b0, mine)) return;
  }
}

// The tiles that are walked: all of them, up to the bound.
template <int STEP>
__device__ __forceinline__ int count_tiles(const GemvW4& p, const unsigned* table) {
  unsigned mine = 0;
  each_32_blocks<STEP>(p, table, [&](int, unsigned tiles) {
    mine = min(mine + tiles, kManyTiles);
    return false;
  });
  const unsigned all = sum_tiles(mine), bound = p.tile_bound;
  if (all > bound && (threadIdx.x & 31) == 0) set_dev_error(SP24_ERR_INVALID_ARG);
  return (int)min(all, bound);
}

// Tile number `tile`, which is below the count.
template <int STEP>
__device__ __forceinline__ TokenTile find_tile(const GemvW4& p, const unsigned* table, unsigned tile) {
  const int lane = threadIdx.x & 31;
  TokenTile t{0, 0, 0};
  // the lane whose tiles the wanted one is among; the tiles before that lane's are taken off
  auto pick = [&](unsigned tiles) {
    const unsigned upto = scan_tiles(tiles);
    const int l = __ffs(__ballot_sync(kFull, upto > tile)) - 1;
    if (l > 0) tile -= __shfl_sync(kFull, upto, l - 1);
    return l;
  };
  each_32_blocks<STEP>(p, table, [&](int b0, unsigned tiles) {
    const unsigned here = sum_tiles(tiles);
    if (tile >= here) {
      tile -= here;
      return false;
    }
    const int e0 = 32 * (b0 + pick(tiles));
    int first, end;
    expert_rows(p, e0 + lane, first, end);
    const int l = pick(tiles_of<STEP>(first, end));
    t = {e0 + l, __shfl_sync(kFull, first, l) + (int)tile * STEP, __shfl_sync(kFull, end, l)};
    return true;
  });
  return t;
}

// The tile after t (there is one).
template <int STEP>
__device__ __forceinline__ TokenTile next_tile(const GemvW4& p, const TokenTile& t) {
  if (t.m0 + STEP < t.m1) return {t.e, t.m0 + STEP, t.m1};
  const int lane = threadIdx.x & 31;
  for (int e = (int)t.e + 1; e < p.E; e += 32) {
    int first, end;
    expert_rows(p, e + lane, first, end);
    const unsigned hit = __ballot_sync(kFull, first < end);
    if (hit) {
      const int l = __ffs(hit) - 1;
      return {e + l, __shfl_sync(kFull, first, l), __shfl_sync(kFull, end, l)};
    }
  }
  return t;  // not reached
}

// Work items are (token tile, column tile) pairs; a team of warps walks a run of them: contiguous with
// experts (column tiles of one expert follow each other), every `teams`-th otherwise (token tiles of
// one column tile follow each other).
template <int STEP>
struct Walk {
  int left;   // items still to come, this one included
  int item;   // without experts
  int col;    // column tile
  TokenTile tok;

  __device__ __forceinline__ void start(const GemvW4& p, const unsigned* table, int col_tiles, int team, int teams) {
    if (p.offsets) {
      const int64_t all = (int64_t)count_tiles<STEP>(p, table) * col_tiles;
      const int64_t first = all * team / teams;
      left = (int)(all * (team + 1) / teams - first);
      if (left <= 0) return;
      col = (int)(first % col_tiles);
      tok = find_tile<STEP>(p, table, (unsigned)(first / col_tiles));
    } else {
      const int tiles = (int)((p.M + STEP - 1) / STEP), all = tiles * col_tiles;
      item = team;
      left = all > team ? (all - team + teams - 1) / teams : 0;
      place(p, tiles);
    }
  }
  __device__ __forceinline__ void place(const GemvW4& p, int tiles) {
    col = tiles == 1 ? item : item / tiles;
    tok = {0, tiles == 1 ? 0 : (item - col * tiles) * STEP, p.M};
  }
  __device__ __forceinline__ void advance(const GemvW4& p, int col_tiles, int teams) {
    if (--left <= 0) return;
    if (p.offsets) {
      if (++col == col_tiles) {
        col = 0;
        tok = next_tile<STEP>(p, tok);
      }
    } else {
      item += teams;
      place(p, (int)((p.M + STEP - 1) / STEP));
    }
  }
  __device__ __forceinline__ int rows() const { return (int)min((int64_t)STEP, tok.m1 - tok.m0); }
};

// y = x W^T for up to 8 NT rows of x and MT tiles of 16 weight rows (with SwiGLU: a gate tile and its
// up tile).  The weight rows are the MMA's M, the rows of x its N.
//
// Persistent, one CTA per SM of four teams, each of which walks work items of its own: one warp
// copies (cp.async, S stages of four chunks of 256 entries ahead, across the items' borders), four
// multiply, each a chunk of every four; mbarriers tell the stages full and empty.  The four chunks
// follow each other along K (WK 4), or, where K has no more than two, pairs of them along the columns
// (WK 2).  The partial sums of the warps that share K meet in shared memory in a fixed order, in two
// buffers that take turns, so one barrier of the team per item is enough.  Where there are few items, the
// four teams take every fourth step of one item's K, and that barrier is the CTA's.
//
// An ldmatrix of 16-byte row pieces hands lane (g, t) the eight codes 8t .. 8t + 7 of a 32-entry block
// of rows g and g + 8; the MMA may sum K in any order, so the pairs that expand8 gives are fed as
// they come, with x's pairs picked alike.  A group's sum is scaled in fp32.
//
// What bounds it: the bytes of codes and scales for large matrices (one token through [151936, 4096],
// groups of 128: 62 us, 5.2 TB/s, 0.79 of the copy rate; 72 us under sustained load, where the power
// limit takes the clock from 1965 to 1732 MHz), with instruction issue behind it: a chunk of 16
// rows, 2 KB, takes about 190 instructions of products proper, and at the copy rate an SM has 88
// cycles for it, so 352 issue slots (54 %).  All instructions together fill 65 % of the slots at 0.7 of
// that rate.  Hence warps of their own for the copies (68 against 74 us with every warp copying
// for itself: no registers are left for its addresses), chunks of 256 instead of 128 entries, expand8
// (74 against 80 us with the codes or-ed into 2^7 and a subtraction), and tables copied per stage of
// four chunks (groups of 32 with zero points: 86 against 146 us with a row's few bytes copied per
// chunk; 92 us now, floor 56).  Small matrices are bound by the launch, the first loads and a warp's own
// latency through its few chunks ([5120, 5120]: 7 us, floor 2.1: its 320 items leave 272 of 592 teams
// without one).  Experts (8 tokens over 10 of 512, SwiGLU, [1024, 2048] each: 23 us, 3.5 TB/s) spend
// half of their instructions between items of two chunks a warp.
//
// A thread has 96 registers, 640 threads in the CTA.  Kernels with x in shared memory fit or spill at most 28
// bytes.  Those with x in global memory, experts among them, store 8 to 132 spilled bytes (32 for SwiGLU
// over experts with groups of 128).
//
// Figures are the GPU's time for a call, in a replayed graph of calls on tensors that take turns.  "a
// against b" is what both forms took side by side when the choice between them was made, a the one that is here.
//
// XW: x stands in shared memory whole, its pairs picked when it is brought there; otherwise (experts,
// or a large x) it is read from global memory half a chunk ahead and its pairs are picked at each use.
//
// Waits are bounded by the library's wait limit, and a warp's lanes give up together.  A multiplying
// warp that gives up records it, does not wait again and passes through the rest of its items, so
// every barrier of its team is still met.  A copying warp records it, waits for its copies in flight
// and ends: it meets no barrier of a team, and the multiplying warps that wait for its next stage give
// up in turn.
template <int XT, int NT, int MT, int S, int WK, bool SWIGLU, bool XW, bool ZEROS, int GB>
struct GemvKernel {
  static constexpr int kTok = 8 * NT;
  static constexpr int kCols = SWIGLU ? 16 : 16 * MT;       // output columns of a warp's tiles
  static constexpr int kSubs = kMulPerTeam / WK;            // of them beside each other in an item
  static constexpr int kItemCols = kCols * kSubs;
  static constexpr int kStep = kChunk * WK;                 // entries of K per stage
  static constexpr int kGroups = kChunk / 32 / GB;          // groups per chunk
  static constexpr int kStepGroups = kGroups * WK;          // and per stage: at least four
  // A stage: four chunks of codes, then the scales and the zero points of its rows.  A row's scales are
  // 2 kStepGroups bytes at any even place, its zero points kStepGroups bytes at any place: the aligned
  // 16-byte pieces that they touch are copied.  The rows of either table are an odd number of pieces
  // apart: eight rows meet no bank twice.
  static constexpr int kRows = 16 * MT * kSubs;
  static constexpr int kScalePieces = (14 + 2 * kStepGroups + 15) / 16, kScaleRow = (kScalePieces | 1) * 16;
  static constexpr int kZeroPieces = (15 + kStepGroups + 15) / 16, kZeroRow = ZEROS ? (kZeroPieces | 1) * 16 : 0;
  static constexpr int kScaleAt = kMulPerTeam * MT * kTileBytes, kZeroAt = kScaleAt + kRows * kScaleRow;
  static constexpr int kStage = (kZeroAt + kRows * kZeroRow + 127) / 128 * 128;
  static constexpr int kPartial = MT * kTok * 16;                               // floats per warp and buffer
  // The front of shared memory: the barriers, then the experts' tile counts.
  static constexpr int kTableAt = 256, kBarriers = 1024;
  static_assert(kTeams * S * 16 <= kTableAt && kTableAt + 4 * kBlocks <= kBarriers);
  static constexpr int kRing = kBarriers + 2 * kMulWarps * kPartial * 4;
  // then 512 zero bytes, at the banks that an odd row of x has, and x
  static constexpr int kZeroX = kRing + kTeams * S * kStage + 64, kFixed = kZeroX + 2 * kChunk + 64;

  static __host__ __device__ __forceinline__ int x_stride(int K) {
    return (2 * K + 127) / 128 * 128 + 64;  // two neighbouring rows of x never meet in a bank
  }
  static int64_t smem_bytes(const GemvW4& p) { return kFixed + (XW ? p.M * x_stride((int)p.K) : 0); }

  static __device__ __forceinline__ void run(const GemvW4& p, uint8_t* smem) {
    // a warp-wide reduction leaves its result where the compiler knows that all lanes agree
    const int warp = (int)__reduce_max_sync(kFull, threadIdx.x >> 5);
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem);  // [team][stage][full, empty]
    if (threadIdx.x == 0) {
      for (int i = 0; i < kTeams * S; ++i) {
        tc::mbar_init(bars + 2 * i, 32);            // every lane of the copying warp
        tc::mbar_init(bars + 2 * i + 1, kMulPerTeam);  // one lane of each multiplying warp
      }
      tc::fence_mbar_init();
    }
    unsigned* const table = reinterpret_cast<unsigned*>(smem + kTableAt);
    begin();
    if (p.offsets)
      for (int b = warp; b < min((int)((p.E + 31) / 32), kBlocks); b += kMulWarps + kTeams) table[b] = block_tiles<kTok>(p, b);
    __syncthreads();
    const bool copies = warp >= kMulWarps;
    const int in_cta = copies ? warp - kMulWarps : warp / kMulPerTeam;
    // teams that share an item walk the same items and take every kTeams-th step of K
    const bool alone = p.share == 1;
    const int team = (alone ? in_cta * gridDim.x : 0) + blockIdx.x, teams = alone ? gridDim.x * kTeams : gridDim.x;
    const int k_first = alone ? 0 : in_cta * kStep, k_step = p.share * kStep;
    uint8_t* const ring = smem + kRing + in_cta * (S * kStage);
    if (copies)
      copy(p, table, ring, bars + 2 * S * in_cta, team, teams, k_first, k_step);
    else
      multiply_all(p, smem, ring, bars + 2 * S * in_cta, warp, in_cta, team, teams, k_first, k_step);
  }

  static __device__ __forceinline__ int64_t columns(const GemvW4& p) { return SWIGLU ? p.N / 2 : p.N; }
  static __device__ __forceinline__ int column_tiles(const GemvW4& p) {
    return (int)((columns(p) + kItemCols - 1) / kItemCols);
  }

  // ---- the copying warp: lane l copies piece l & 7 of rows (l >> 3) + 4 h of each of the four chunks
  static __device__ __forceinline__ void copy(const GemvW4& p, const unsigned* table, uint8_t* ring, uint64_t* bars, int team,
                                              int teams, int k_first, int k_step) {
    const int lane = threadIdx.x & 31;
    const int64_t cols = columns(p);
    const int col_tiles = column_tiles(p);
    const int K = (int)p.K, KG = K / (32 * GB);
    const int64_t groups_total = p.E * p.N * KG;
    const uint8_t* const scales = reinterpret_cast<const uint8_t*>(p.scales);
    const uint32_t ring_at = smem_addr(ring);
    // a row's pieces change places by its number: row r's piece i stands at i ^ (r & 7)
    const uint32_t code_at = ring_at + (lane >> 3) * 128 + 16 * ((lane & 7) ^ (lane >> 3));  // h odd: ^ 64
    Walk<kTok> walk;
    walk.start(p, table, col_tiles, team, teams);
    int stage = 0, round = 0;
    int64_t near_row = -1;  // first row of x of the tile that was last brought to L1
    for (; walk.left > 0; walk.advance(p, col_tiles, teams)) {
      if (!XW && walk.tok.m0 != near_row) {  // x of a new token tile: into L1 ahead of the multiplying warps
        near_row = walk.tok.m0;
        const uint8_t* const x = reinterpret_cast<const uint8_t*>(p.x) + near_row * K * 2;
        for (int64_t at = 128 * lane; at < (int64_t)walk.rows() * K * 2; at += 128 * 32)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(x + at));
      }
      const int left = (int)min((int64_t)kItemCols, cols - (int64_t)walk.col * kItemCols);  // columns of this item
      const int64_t row0 = walk.tok.e * p.N + (int64_t)walk.col * kItemCols;
      // a copied piece may reach past the arrays' ends: a stage may name groups past a row's last
      const bool near_end = row0 + (SWIGLU ? cols : 0) + kItemCols + kStepGroups + 16 >= p.E * p.N;
      const uint8_t* code_src[MT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 4; ++h)
          code_src[i][h] =
              p.codes + (row0 + (SWIGLU ? i * cols : 16 * i) + (lane >> 3) + 4 * h) * (K / 2) + 16 * (lane & 7) + k_first / 2;
      // the first group of table row r's weight row: of the item's first row, and from there on
      const int64_t base0 = row0 * KG, base1 = SWIGLU ? (row0 + cols) * KG : base0;
      auto base = [&](int r) { return SWIGLU && (r & 16) ? base1 : base0; };
      auto row_of = [&](int r) { return SWIGLU ? (r & 15) + (r >> 5) * 16 : r; };  // within the item

      for (int k0 = k_first; k0 < K; k0 += k_step) {
        if (round && !warp_wait(bars + 2 * stage + 1, (round - 1) & 1)) {
          set_dev_error(SP24_ERR_DEVICE_TIMEOUT);
          copy_wait_all();
          return;
        }
        const uint32_t dst = code_at + stage * kStage;
        if (left == kItemCols && k0 + kStep <= K) {
#pragma unroll
          for (int c = 0; c < kMulPerTeam; ++c) {
            const int64_t on = c % WK * (kChunk / 2) + (c < WK ? 0 : (int64_t)(c / WK * kCols) * (K / 2));
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int h = 0; h < 4; ++h)
                copy16((h & 1 ? dst ^ 64 : dst) + ((c * MT + i) * kTileBytes + h * 512), code_src[i][h] + on);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < kMulPerTeam; ++c) {
            const int col = c / WK * kCols;
            const int64_t on = c % WK * (kChunk / 2) + (int64_t)col * (K / 2);
            if (k0 + c % WK * kChunk + 32 * (lane & 7) < K)
#pragma unroll
              for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 4; ++h)
                  if (col + (SWIGLU ? 0 : 16 * i) + (lane >> 3) + 4 * h < left)
                    copy16((h & 1 ? dst ^ 64 : dst) + ((c * MT + i) * kTileBytes + h * 512), code_src[i][h] + on);
          }
        }
        const int g0 = k0 / (32 * GB);
        const uint32_t scale_at = ring_at + stage * kStage + kScaleAt, zero_at = ring_at + stage * kStage + kZeroAt;
#pragma unroll
        for (int s0 = 0; s0 < kRows * kScalePieces; s0 += 32) {
          const int s = s0 + lane, r = s / kScalePieces, q = s % kScalePieces;
          const int64_t b = base(r);
          const int at = ((int)b & 7) + row_of(r) * KG + g0;  // in scales, from the piece that b is in
          if (s < kRows * kScalePieces && row_of(r) < left && 8 * q < (at & 7) + kStepGroups) {
            const uint8_t* const src = scales + (b >> 3) * 16 + ((at >> 3) + q) * 16;
            if (near_end)
              copy16(scale_at + r * kScaleRow + 16 * q, src, scales + 2 * groups_total, scales);
            else
              copy16(scale_at + r * kScaleRow + 16 * q, src);
          }
        }
        if constexpr (ZEROS) {
#pragma unroll
          for (int s0 = 0; s0 < kRows * kZeroPieces; s0 += 32) {
            const int s = s0 + lane, r = s / kZeroPieces, q = s % kZeroPieces;
            const int64_t b = base(r);
            const int at = ((int)b & 15) + row_of(r) * KG + g0;
            if (s < kRows * kZeroPieces && row_of(r) < left && 16 * q < (at & 15) + kStepGroups) {
              const uint8_t* const src = p.zeros + (b >> 4) * 16 + ((at >> 4) + q) * 16;
              if (near_end)
                copy16(zero_at + r * kZeroRow + 16 * q, src, p.zeros + groups_total, p.zeros);
              else
                copy16(zero_at + r * kZeroRow + 16 * q, src);
            }
          }
        }
        copy_arrive(bars + 2 * stage);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int h = 0; h < 4; ++h) code_src[i][h] += k_step / 2;
        if (++stage == S) stage = 0, ++round;
      }
    }
    copy_wait_all();
  }

  // ---- a multiplying warp
  static __device__ __forceinline__ void multiply_all(const GemvW4& p, uint8_t* smem, uint8_t* ring, uint64_t* bars,
                                                      int warp, int in_cta, int team, int teams, int k_first, int k_step) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int in_team = warp & (kMulPerTeam - 1), kw = in_team % WK, sub = in_team / WK;
    const int64_t cols = columns(p);
    const int col_tiles = column_tiles(p);
    const int K = (int)p.K, KG = K / (32 * GB);
    float* const partials = reinterpret_cast<float*>(smem + kBarriers);  // [buffer][warp][tile][token][row]
    uint8_t* const x_all = smem + kFixed;
    if (XW) {
      if (threadIdx.x < 2 * kChunk / 16) reinterpret_cast<uint4*>(smem + kZeroX)[threadIdx.x] = make_uint4(0, 0, 0, 0);
      const int pieces = K / 8;
      for (int j = threadIdx.x; j < pieces; j += 32 * kMulWarps) {
        uint4 v[kTok];  // every row's loads in flight together
#pragma unroll
        for (int m = 0; m < kTok; ++m)
          if (m < (int)p.M) v[m] = reinterpret_cast<const uint4*>(p.x)[(int64_t)m * pieces + j];
#pragma unroll
        for (int m = 0; m < kTok; ++m)
          if (m < (int)p.M)
            *reinterpret_cast<uint4*>(x_all + m * x_stride(K) + 16 * j) =
                make_uint4(__byte_perm(v[m].x, v[m].z, 0x5410), __byte_perm(v[m].x, v[m].z, 0x7632),
                           __byte_perm(v[m].y, v[m].w, 0x5410), __byte_perm(v[m].y, v[m].w, 0x7632));
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + kTeams), "r"(32 * kMulWarps) : "memory");
    }

    Walk<kTok> walk;
    walk.start(p, reinterpret_cast<const unsigned*>(smem + kTableAt), col_tiles, team, teams);
    // ldmatrix: lane l names row (l & 7) + 8 (l >> 3 & 1) of block (l >> 4); block j + 2 n: ^ 32 n
    const int lm_row = (lane & 7) + 8 * (lane >> 3 & 1);
    const uint32_t lm_at = smem_addr(ring) + in_team * (MT * kTileBytes) + lm_row * 128 + 16 * ((lane >> 4) ^ (lane & 7));
    const uint8_t* const scale_row = ring + kScaleAt + (sub * 16 * MT + g) * kScaleRow + 2 * kw * kGroups;
    const uint8_t* const zero_row = ring + kZeroAt + (sub * 16 * MT + g) * kZeroRow + kw * kGroups;
    float tot[MT][NT][4], acc[MT][NT][4];

    // x of kAhead blocks of the chunk at entry k, as it stands in memory, read one such part ahead
    constexpr int kAhead = 4, kParts = kChunk / 32 / kAhead;
    // This lane's rows of x.  Columns past the last row are not stored.  With x in shared memory they are 0:
    // the MMA draws less power so, and power is what limits the clock.  Otherwise they repeat the last row
    // (zeros there, over experts: 25.3 against 24.8 us).
    const uint8_t* x_row[NT];
    int x_on[NT];
    // Where the first group of this lane's row of tile i stands within a piece, in bytes; a further stage
    // moves that on unless its groups fill pieces.
    int scale_odd[MT], zero_odd[MT];
    auto read_x = [&](uint4 (&xv)[NT][kAhead], int k, int part, int blocks) {
      if constexpr (!XW)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            if (kAhead * part + j < blocks)
              xv[n][j] = *reinterpret_cast<const uint4*>(x_row[n] + 2 * k + 64 * (kAhead * part + j));
    };
    // blocks j, j + 1 of the chunk in the stage
    auto multiply2 = [&](uint32_t stage, int k, int j, const uint4 (&xv)[NT][kAhead], bool both) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint32_t words[4];
        ldmatrix4(words, (lm_at ^ (16 * j)) + stage + i * kTileBytes);
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
          if (jb && !both) break;
          const int jj = j + jb;
          uint32_t zl = Expand<XT>::zero(8), zh = zl;
          if (ZEROS) {  // eight rows on, an odd KG moves the place by eight bytes
            const uint8_t* zp = zero_row + stage + 16 * i * kZeroRow + jj / GB;
            const int l = zero_odd[i] + (kStepGroups % 16 ? (k - kw * kChunk) / (32 * GB) : 0), h = l + 8 * (KG & 1);
            zl = Expand<XT>::zero_of(zp[l & 15]);
            zh = Expand<XT>::zero_of(zp[8 * kZeroRow + (h & 15)]);
          }
          uint32_t lo[4], hi[4];
          expand8<XT>(words[2 * jb], zl, lo);
          expand8<XT>(words[2 * jb + 1], zh, hi);
          const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint4 b;
            if constexpr (XW) {
              b = *reinterpret_cast<const uint4*>(x_row[n] + (2 * k & x_on[n]) + 64 * jj);
            } else {
              b = xv[n][jj % kAhead];
              b = make_uint4(__byte_perm(b.x, b.z, 0x5410), __byte_perm(b.x, b.z, 0x7632), __byte_perm(b.y, b.w, 0x5410),
                             __byte_perm(b.y, b.w, 0x7632));
            }
            if (jj % GB == 0)
              mma16816_first<XT>(acc[i][n], a0, b.x, b.y);
            else
              mma16816<XT>(acc[i][n], a0, b.x, b.y);
            mma16816<XT>(acc[i][n], a1, b.z, b.w);
          }
          if ((jj + 1) % GB == 0) {
            const int from = kStepGroups % 8 ? (scale_odd[i] + (k - kw * kChunk) / (16 * GB)) & 15 : scale_odd[i];
            const uint8_t* sp = scale_row + stage + from + 16 * i * kScaleRow + 2 * (jj / GB);
            const uint32_t l = *reinterpret_cast<const uint16_t*>(sp);
            const uint32_t h = *reinterpret_cast<const uint16_t*>(sp + 8 * kScaleRow);
            const float sl = p.scale_dtype == SP24_BF16 ? W4Half<SP24_BF16>::get(l) : W4Half<SP24_F16>::get(l);
            const float sh = p.scale_dtype == SP24_BF16 ? W4Half<SP24_BF16>::get(h) : W4Half<SP24_F16>::get(h);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int k = 0; k < 4; ++k) tot[i][n][k] = fmaf(k < 2 ? sl : sh, acc[i][n][k], tot[i][n][k]);
          }
        }
      }
    };
    auto multiply = [&](uint32_t stage, int k, const uint4 (&xv)[NT][kAhead], int part, int blocks) {
#pragma unroll
      for (int j = kAhead * part; j < kAhead * (part + 1); j += 2)
        if (j < blocks) multiply2(stage, k, j, xv, j + 1 < blocks);
    };

    int stage = 0, parity = 0, buffer = 0;
    bool given_up = false;
    for (; walk.left > 0; walk.advance(p, col_tiles, teams)) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        // rows 8 on, and further tiles of 16: the same place of a scale
        const int64_t row = walk.tok.e * p.N + (SWIGLU ? i * cols : 0) + (int64_t)walk.col * kItemCols + g;
        scale_odd[i] = ((int)(row & 7) * KG & 7) * 2;
        zero_odd[i] = (int)(row & 15) * KG & 15;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) tot[i][n][k] = 0.0f;
      }
      const int rows = walk.rows();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int m = 8 * n + g;
        x_on[n] = m < rows ? -1 : 0;
        if (XW)
          x_row[n] = (m < rows ? x_all + m * x_stride(K) : smem + kZeroX) + 16 * t;
        else
          x_row[n] = reinterpret_cast<const uint8_t*>(p.x) + ((walk.tok.m0 + min(m, rows - 1)) * K + 8 * t) * 2;
      }
      for (int k = k_first + kw * kChunk; k < K + kw * kChunk; k += k_step) {  // every warp meets every stage
        const int blocks = min(kChunk / 32, (K - k) / 32);
        const uint32_t at = stage * kStage;
        uint4 x[2][NT][kAhead];
        read_x(x[0], k, 0, blocks);
        if (!given_up && !warp_wait(bars + 2 * stage, parity)) {
          set_dev_error(SP24_ERR_DEVICE_TIMEOUT);
          given_up = true;
        }
        if (blocks == kChunk / 32) {  // a whole chunk: straight through
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            if (part + 1 < kParts) read_x(x[(part + 1) & 1], k, part + 1, kChunk / 32);
            multiply(at, k, x[part & 1], part, kChunk / 32);
          }
        } else if (blocks > 0) {
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            multiply(at, k, x[0], part, blocks);
            if (part + 1 < kParts) read_x(x[0], k, part + 1, blocks);
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bars + 2 * stage + 1);
        if (++stage == S) stage = 0, parity ^= 1;
      }

      float* const mine = partials + (buffer * kMulWarps + warp) * kPartial;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int m = 8 * n + 2 * t + (k & 1);
            if (m < rows) mine[(i * kTok + m) * 16 + g + 8 * (k >> 1)] = tot[i][n][k] * (1.0f / Expand<XT>::kUnit);
          }
      const bool alone = p.share == 1;
      if (alone)
        asm volatile("bar.sync %0, %1;" ::"r"(1 + in_cta), "r"(32 * kMulPerTeam) : "memory");
      else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + kTeams), "r"(32 * kMulWarps) : "memory");
      const float* const sums = partials + (buffer * kMulWarps + (alone ? in_cta * kMulPerTeam : 0)) * kPartial;
      constexpr int kOutTiles = SWIGLU ? 1 : MT;
      constexpr int kTiles = kItemCols / 16;
      for (int o = (alone ? in_team : warp) * 32 + lane; o < rows * kTiles * 16; o += p.share * 32 * kMulPerTeam) {
        const int r = o & 15, tile = (o >> 4) % kTiles, m = (o >> 4) / kTiles;
        const int64_t col = (int64_t)walk.col * kItemCols + 16 * tile + r;
        if (col >= cols) continue;
        const int i = tile % kOutTiles, first = tile / kOutTiles * WK;
        float v = 0.0f, up = 0.0f;
        auto add = [&](const float* from) {
#pragma unroll
          for (int k = 0; k < WK; ++k) {
            v += from[k * kPartial + (i * kTok + m) * 16 + r];
            if (SWIGLU) up += from[k * kPartial + (kTok + m) * 16 + r];
          }
        };
        add(sums + first * kPartial);
        if (!alone)
          for (int q = 1; q < kTeams; ++q) add(sums + (q * kMulPerTeam + first) * kPartial);
        if (SWIGLU) v = v / (1.0f + expf(-v)) * up;
        const int64_t out = (walk.tok.m0 + m) * cols + col;
        if (p.y_f32)
          reinterpret_cast<float*>(p.y)[out] = v;
        else
          reinterpret_cast<uint16_t*>(p.y)[out] = (uint16_t)W4Half<XT>::put(v);
      }
      buffer ^= 1;
    }
  }
};

template <int XT, int NT, int MT, int S, int WK, bool SWIGLU, bool XW, bool ZEROS, int GB>
__global__ void __launch_bounds__(32 * (kMulWarps + kTeams), 1) gemv_w4_kernel(const __grid_constant__ GemvW4 p) {
  extern __shared__ __align__(128) uint8_t smem[];
  GemvKernel<XT, NT, MT, S, WK, SWIGLU, XW, ZEROS, GB>::run(p, smem);
}

template <int XT, int NT, int MT, int S, int WK, bool SWIGLU, bool XW, bool ZEROS, int GB>
int launch_gemv(GemvW4 p, cudaStream_t s) {
  using Kern = GemvKernel<XT, NT, MT, S, WK, SWIGLU, XW, ZEROS, GB>;
  auto kernel = gemv_w4_kernel<XT, NT, MT, S, WK, SWIGLU, XW, ZEROS, GB>;
  static std::atomic<bool> raised[64];  // the attribute holds per device; threads may set it twice
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SP24_ERR_CUDA;
  if (!raised[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
      return SP24_ERR_CUDA;
    raised[dev].store(true, std::memory_order_relaxed);
  }
  const int64_t cols = SWIGLU ? p.N / 2 : p.N, col_tiles = (cols + Kern::kItemCols - 1) / Kern::kItemCols;
  // with experts: the sum of ceil(rows / kTok) is at most this
  const int64_t tok_tiles = (p.M + Kern::kTok - 1) / Kern::kTok + (p.offsets ? (p.E < p.M ? p.E : p.M) : 0);
  const int64_t items = col_tiles * tok_tiles;
  if (items > INT32_MAX / 2) return SP24_ERR_UNSUPPORTED;
  p.tile_bound = (int)tok_tiles;
  // Few items: the four teams of a CTA take the K of one together.  The cost is rounds of items times
  // steps of K and about one for an item's ends (12 rows through [48, 11232], groups of 32 with zero
  // points: 15 us shared, 23 alone).
  const int sms = sm_count();
  const int64_t steps = (p.K + Kern::kStep - 1) / Kern::kStep;
  const int64_t alone = (items + kTeams * sms - 1) / (kTeams * sms) * (steps + 1);
  const int64_t shared = (items + sms - 1) / sms * ((steps + kTeams - 1) / kTeams + 1);
  p.share = shared < alone ? kTeams : 1;
  const int64_t ctas = items < sms ? items : sms;
  return launch_after(kernel, (unsigned)ctas, 32 * (kMulWarps + kTeams), (size_t)Kern::smem_bytes(p), s, p);
}

template <int XT, int NT, int MT, int S, int WK, bool SWIGLU, bool XW>
int by_group(const GemvW4& p, cudaStream_t s) {
  if (p.zeros) {
    if (p.group == 128) return launch_gemv<XT, NT, MT, S, WK, SWIGLU, XW, true, 4>(p, s);
    if (p.group == 64) return launch_gemv<XT, NT, MT, S, WK, SWIGLU, XW, true, 2>(p, s);
    return launch_gemv<XT, NT, MT, S, WK, SWIGLU, XW, true, 1>(p, s);
  }
  if (p.group == 128) return launch_gemv<XT, NT, MT, S, WK, SWIGLU, XW, false, 4>(p, s);
  if (p.group == 64) return launch_gemv<XT, NT, MT, S, WK, SWIGLU, XW, false, 2>(p, s);
  return launch_gemv<XT, NT, MT, S, WK, SWIGLU, XW, false, 1>(p, s);
}

// x as a whole in shared memory where it fits beside the ring, and is one tile's rows of one matrix
// (one and eight rows through [151936, 4096]: 62 and 64 us, against 69 and 79 us read from global memory;
// through [5120, 5120]: 7.0 and 8.1 against 9.5 and 10.5 us).
template <int XT, int NT, int MT, int S, int WK, bool SWIGLU>
bool x_fits(const GemvW4& p) {
  using Kern = GemvKernel<XT, NT, MT, S, WK, SWIGLU, true, true, 1>;  // the largest stages
  return !p.offsets && p.M <= Kern::kTok && p.M * (int64_t)Kern::x_stride((int)p.K) <= kSmemMax - Kern::kFixed;
}

// A K of no more than two chunks leaves two of four warps along K without work: those go along the
// columns instead ([160000, 512]: 15 against 27 us).  A third stage is worth 2 % (64 against 65.5 us above)
// and given up for an x that then fits (4 rows of 16384: 8.8 against 14 us through [300, 16384]).  Nine to sixteen rows share a tile where their x
// fits shared memory (12 rows through [16384, 2048]: 8.5 us, against 12.3 us as two tiles); where it does
// not, two tiles of eight are faster (16 rows through [75000, 4096]: 82 against 89 us).
template <int XT>
int gemv_w4_plain(const GemvW4& p, cudaStream_t s) {
  if (p.K <= 2 * kChunk)
    return x_fits<XT, 1, 1, 3, 2, false>(p) ? by_group<XT, 1, 1, 3, 2, false, true>(p, s)
                                            : by_group<XT, 1, 2, 2, 2, false, false>(p, s);
  if (x_fits<XT, 1, 1, 3, 4, false>(p)) return by_group<XT, 1, 1, 3, 4, false, true>(p, s);
  if (x_fits<XT, 1, 1, 2, 4, false>(p)) return by_group<XT, 1, 1, 2, 4, false, true>(p, s);
  return x_fits<XT, 2, 1, 2, 4, false>(p) ? by_group<XT, 2, 1, 2, 4, false, true>(p, s)
                                          : by_group<XT, 1, 2, 2, 4, false, false>(p, s);
}

template <int XT>
int gemv_w4_swiglu(const GemvW4& p, cudaStream_t s) {
  if (p.K <= 2 * kChunk)
    return x_fits<XT, 1, 2, 2, 2, true>(p) ? by_group<XT, 1, 2, 2, 2, true, true>(p, s)
                                           : by_group<XT, 1, 2, 2, 2, true, false>(p, s);
  return x_fits<XT, 1, 2, 2, 4, true>(p) ? by_group<XT, 1, 2, 2, 4, true, true>(p, s)
                                         : by_group<XT, 1, 2, 2, 4, true, false>(p, s);
}

}  // namespace
}  // namespace sp24
