// The kernel of sp24_gemv_w4 / sp24_gemv_w4_grouped; each type of x is a translation unit of its own.
#pragma once

#include "sp24_w4.cuh"

namespace sp24 {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kChunk = 128;     // entries of K per stage: 64 code bytes of each row
constexpr int kTileBytes = 16 * kChunk / 2;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src));
}
// The four bytes at byte `at` (a multiple of 4) of an array of `total` bytes; zeros past its end.
__device__ __forceinline__ void copy4(uint32_t dst, const void* base, int64_t at, int64_t total) {
  const int n = at + 4 <= total ? 4 : at < total ? (int)(total - at) : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst),
               "l"(reinterpret_cast<const uint8_t*>(base) + (n ? at : 0)), "r"(n));
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N));
}
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

// The code q as a 16-bit float without a conversion: its four bits are or-ed into the significand of
// 2^10 (f16) or 2^7 (bf16), whose last place is 1, and the same number plus the zero point is
// subtracted: q - z exactly.  kMagic is that number's bits, in both halves of a word.
template <int XT>
constexpr uint32_t kMagic = XT == SP24_BF16 ? 0x43004300u : 0x64006400u;

// (word & mask) | magic, one three-input logic operation.
__device__ __forceinline__ uint32_t and_or(uint32_t word, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(word), "r"(mask), "r"(magic));
  return r;
}

template <int XT>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  if (XT == SP24_BF16) {
    const __nv_bfloat162 r = __hsub2(reinterpret_cast<const __nv_bfloat162&>(a), reinterpret_cast<const __nv_bfloat162&>(b));
    return reinterpret_cast<const uint32_t&>(r);
  }
  const __half2 r = __hsub2(reinterpret_cast<const __half2&>(a), reinterpret_cast<const __half2&>(b));
  return reinterpret_cast<const uint32_t&>(r);
}

// The eight codes of a word as four pairs of q - z: entries (0, 4), (1, 5), (2, 6), (3, 7).  `zero` is
// kMagic + z in both halves.
template <int XT>
__device__ __forceinline__ void expand8(uint32_t word, uint32_t zero, uint32_t (&out)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) out[k] = sub2<XT>(and_or(word >> (4 * k), 0x000f000fu, kMagic<XT>), zero);
}

// The token tiles of all experts, in expert order: expert e has ceil(rows of e / step) of them.
// Everything here is computed by a whole warp together.
struct TokenTile {
  int64_t e, m0, m1;  // expert, first row, end of the expert's rows
};

__device__ __forceinline__ int64_t expert_rows(const GemvW4& p, int64_t e, int64_t& first, int64_t& end) {
  first = max(0, p.offsets[e]);
  end = min(p.M, (int64_t)p.offsets[e + 1]);
  return max((int64_t)0, end - first);
}

__device__ __forceinline__ int64_t warp_scan(int64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(kFull, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// The number of token tiles; lane l's run of ceil(E / 32) experts has those before `upto`.
__device__ __forceinline__ int64_t count_tiles(const GemvW4& p, int step, int64_t& mine, int64_t& upto) {
  const int lane = threadIdx.x & 31;
  const int64_t per = (p.E + 31) / 32;
  int64_t a, b;
  mine = 0;
  for (int64_t i = lane * per; i < min(p.E, (lane + 1) * per); ++i) mine += (expert_rows(p, i, a, b) + step - 1) / step;
  upto = warp_scan(mine);
  return __shfl_sync(kFull, upto, 31);
}

// Tile number `tile`, given count_tiles' values.
__device__ __forceinline__ TokenTile find_tile(const GemvW4& p, int step, int64_t mine, int64_t upto, int64_t tile) {
  const int lane = threadIdx.x & 31;
  const int64_t per = (p.E + 31) / 32;
  const int who = __ffs(__ballot_sync(kFull, upto > tile)) - 1;
  tile -= __shfl_sync(kFull, upto - mine, who);
  const int64_t end = min(p.E, (who + 1) * per);
  for (int64_t i0 = who * per; i0 < end; i0 += 32) {
    int64_t a = 0, b = 0;
    const int64_t n = i0 + lane < end ? (expert_rows(p, i0 + lane, a, b) + step - 1) / step : 0;
    const int64_t s = warp_scan(n);
    const unsigned hit = __ballot_sync(kFull, s > tile);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int64_t first = __shfl_sync(kFull, a, l), before = __shfl_sync(kFull, s - n, l);
      return {i0 + l, first + (tile - before) * step, __shfl_sync(kFull, b, l)};
    }
    tile -= __shfl_sync(kFull, s, 31);
  }
  return {0, 0, 0};  // not reached: tile is below the count
}

// The tile after t (there is one).
__device__ __forceinline__ TokenTile next_tile(const GemvW4& p, int step, const TokenTile& t) {
  if (t.m0 + step < t.m1) return {t.e, t.m0 + step, t.m1};
  const int lane = threadIdx.x & 31;
  for (int64_t e = t.e + 1; e < p.E; e += 32) {
    int64_t a = 0, b = 0;
    const bool some = e + lane < p.E && expert_rows(p, e + lane, a, b) > 0;
    const unsigned hit = __ballot_sync(kFull, some);
    if (hit) {
      const int l = __ffs(hit) - 1;
      return {e + l, __shfl_sync(kFull, a, l), __shfl_sync(kFull, b, l)};
    }
  }
  return t;  // not reached
}

// Work items are (token tile, column tile) pairs.  A CTA walks a run of them: contiguous with
// experts (column tiles of one expert follow each other), every gridDim.x-th otherwise (token tiles
// of one column tile follow each other).
template <int STEP>
struct Walk {
  int64_t left;       // items still to come, this one included
  int64_t item;       // without experts
  int64_t col;        // column tile
  TokenTile tok;

  __device__ __forceinline__ void start(const GemvW4& p, int64_t col_tiles) {
    const int64_t cta = blockIdx.x, ctas = gridDim.x;
    if (p.offsets) {
      int64_t mine, upto;
      const int64_t all = count_tiles(p, STEP, mine, upto) * col_tiles;
      const int64_t first = all * cta / ctas;
      left = all * (cta + 1) / ctas - first;
      if (left <= 0) return;
      col = first % col_tiles;
      tok = find_tile(p, STEP, mine, upto, first / col_tiles);
    } else {
      const int64_t tiles = (p.M + STEP - 1) / STEP, all = tiles * col_tiles;
      item = cta;
      left = all > cta ? (all - cta + ctas - 1) / ctas : 0;
      place(p, tiles);
    }
  }
  __device__ __forceinline__ void place(const GemvW4& p, int64_t tiles) {
    col = tiles == 1 ? item : item / tiles;
    tok = {0, tiles == 1 ? 0 : (item - col * tiles) * STEP, p.M};
  }
  __device__ __forceinline__ void advance(const GemvW4& p, int64_t col_tiles) {
    if (--left <= 0) return;
    if (p.offsets) {
      if (++col == col_tiles) {
        col = 0;
        tok = next_tile(p, STEP, tok);
      }
    } else {
      item += gridDim.x;
      place(p, (p.M + STEP - 1) / STEP);
    }
  }
  __device__ __forceinline__ int rows() const { return (int)min((int64_t)STEP, tok.m1 - tok.m0); }
};

// y = x W^T for up to 8 NT rows of x and MT tiles of 16 weight rows per warp (with SwiGLU: a gate
// tile and its up tile).  The weight rows are the MMA's M, the rows of x its N.
//
// Persistent: a CTA walks its work items with the loads running S chunks ahead across their borders.
// K is split over wk warps of the CTA in chunks of 128 entries; each warp streams its chunks of codes
// through a ring of S stages of its own with cp.async, so within an item no warp waits for another.
// An ldmatrix of 16-byte row pieces hands lane (g, t) the eight codes 8t .. 8t + 7 of a 32-entry
// block of rows g and g + 8; the MMA may sum K in any order, so the pairs that expand8 gives are fed
// as they come, with x's pairs picked alike.  A group's sum is scaled in fp32; the warps' partial
// sums meet in shared memory in a fixed order, in two buffers that take turns, so one barrier per
// item is enough.
//
// XW: x stands in shared memory whole, its pairs picked when it is brought there (few rows of x, one
// matrix); otherwise its chunk travels in the ring and the pairs are picked at each use.
template <int XT, int NT, int MT, int S, bool SWIGLU, bool XW, bool ZEROS, int GB>
struct GemvKernel {
  static constexpr int kTok = 8 * NT;
  static constexpr int kCols = SWIGLU ? 16 : 16 * MT;    // output columns per warp
  static constexpr int kGroups = 4 / GB;                 // groups per chunk
  // A chunk's scales of one row are 2 kGroups bytes at any even place, its zero points kGroups bytes
  // at any place: the aligned words that they may touch are copied.
  static constexpr int kScaleWords = kGroups / 2 + 1;
  static constexpr int kZeroWords = ZEROS ? (kGroups == 1 ? 1 : 2) : 0;
  static constexpr int kZeroAt = 16 * MT * kScaleWords * 4;                     // in bytes, behind the scales
  static constexpr int kScaleBytes = kZeroAt + 16 * MT * kZeroWords * 4;
  static constexpr int kPartial = kWarps * MT * kTok * 16;       // floats of one buffer

  static __host__ __device__ __forceinline__ int stage_bytes(int x_rows) {
    return MT * kTileBytes + kScaleBytes + (XW ? 0 : x_rows * 2 * kChunk);
  }
  static __host__ __device__ __forceinline__ int x_stride(int K) {
    return (2 * K + 127) / 128 * 128 + 64;  // two neighbouring rows of x never meet in a bank
  }
  static int64_t smem_bytes(const GemvW4& p) {
    return 2 * kPartial * 4 + (int64_t)kWarps * S * stage_bytes(p.x_rows) + (XW ? p.x_rows * x_stride((int)p.K) : 0);
  }

  static __device__ __forceinline__ void run(const GemvW4& p, uint8_t* smem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int wk = p.wk, wn = kWarps / wk;
    const int kw = warp & (wk - 1), nw = warp / wk;
    const int64_t cols = SWIGLU ? p.N / 2 : p.N;
    const int64_t col_tiles = (cols + kCols * wn - 1) / (kCols * wn);
    const int K = (int)p.K, KG = K / (32 * GB);
    const int chunks = (K + kChunk - 1) / kChunk;

    const int stage_size = stage_bytes(p.x_rows);
    float* partial = reinterpret_cast<float*>(smem);
    uint8_t* ring = smem + 2 * kPartial * 4 + warp * S * stage_size;
    uint8_t* x_all = smem + 2 * kPartial * 4 + kWarps * S * stage_size;
    const uint32_t ring_at = smem_addr(ring);

    Walk<kTok> load, use;  // what is being fetched and what is being multiplied
    load.start(p, col_tiles);
    if (load.left <= 0) return;
    use = load;

    // ---- fetching: chunk load_c of the item `load`
    int load_c = kw;
    const uint8_t* code_src[MT][2];
    const uint8_t* x_src = nullptr;
    const int64_t groups_total = p.E * p.N * KG;
    int64_t row_group[(16 * MT * kScaleWords + 31) / 32];  // first group of the rows whose words this lane copies
    int64_t row_group_z[(16 * MT * (ZEROS ? kZeroWords : 1) + 31) / 32];
    int load_rows = 0;
    auto aim = [&]() {  // the sources of a new item
      const int64_t col0 = (load.col * wn + nw) * kCols;
      auto weight_row = [&](int i, int r) {  // past the end: the last row, computed and not stored
        const int64_t c = min(col0 + (SWIGLU ? r : 16 * i + r), cols - 1);
        return load.tok.e * p.N + (SWIGLU ? i * cols : 0) + c;
      };
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          code_src[i][h] = p.codes + weight_row(i, g + 8 * h) * (p.K / 2) + 16 * t + kw * (kChunk / 2);
#pragma unroll
      for (int i = 0; 32 * i < 16 * MT * kScaleWords; ++i) {
        const int r = (lane + 32 * i) / kScaleWords;
        row_group[i] = weight_row(r >> 4 & (MT - 1), r & 15) * KG + kw * kGroups;
      }
#pragma unroll
      for (int i = 0; 32 * i < 16 * MT * kZeroWords; ++i) {
        const int r = (lane + 32 * i) / (ZEROS ? kZeroWords : 1);
        row_group_z[i] = weight_row(r >> 4 & (MT - 1), r & 15) * KG + kw * kGroups;
      }
      if (!XW) {
        x_src = reinterpret_cast<const uint8_t*>(p.x) + load.tok.m0 * p.K * 2;
        load_rows = load.rows();
      }
    };
    const uint32_t code_dst = ring_at + g * 64 + 16 * (t ^ (g >> 1 & 3));  // rows g and g + 8 swizzle alike
    auto fetch = [&](int slot) {
      if (load.left > 0) {
        const int k0 = load_c * kChunk;
        const uint32_t dst = code_dst + slot * stage_size;
        if (k0 + 32 * t < K) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) copy16(dst + i * kTileBytes + h * 512, code_src[i][h]);
        }
        const uint32_t table = ring_at + slot * stage_size + MT * kTileBytes;
#pragma unroll
        for (int i = 0; 32 * i < 16 * MT * kScaleWords; ++i) {
          const int s = lane + 32 * i, w = s % kScaleWords;
          const int64_t at = row_group[i];
          if (s < 16 * MT * kScaleWords && 2 * w < (at & 1) + kGroups)
            copy4(table + 4 * s, p.scales, (at >> 1) * 4 + 4 * w, 2 * groups_total);
          row_group[i] += wk * kGroups;
        }
#pragma unroll
        for (int i = 0; 32 * i < 16 * MT * kZeroWords; ++i) {
          const int s = lane + 32 * i, w = s % (ZEROS ? kZeroWords : 1);
          const int64_t at = row_group_z[i];
          if (s < 16 * MT * kZeroWords && 4 * w < (at & 3) + kGroups)
            copy4(table + kZeroAt + 4 * s, p.zeros, (at >> 2) * 4 + 4 * w, groups_total);
          row_group_z[i] += wk * kGroups;
        }
        if (!XW) {  // x: row m's 256 bytes at 256 m, its 16-byte piece j at 16 (j ^ 4 (m & 1))
          const uint32_t xdst = ring_at + slot * stage_size + MT * kTileBytes + kScaleBytes;
          for (int j = lane; j < load_rows * 16; j += 32) {
            const int m = j >> 4, piece = j & 15;
            if (k0 + 8 * piece < K)
              copy16(xdst + m * 256 + 16 * (piece ^ (m & 1) * 4), x_src + ((int64_t)m * K + k0 + 8 * piece) * 2);
          }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) code_src[i][h] += wk * (kChunk / 2);
        load_c += wk;
        if (load_c >= chunks) {
          load.advance(p, col_tiles);
          load_c = kw;
          if (load.left > 0) aim();
        }
      }
      copy_commit();
    };
    aim();
#pragma unroll
    for (int s = 0; s < S; ++s) fetch(s);
    if (XW) {
      const int pieces = K / 8, rows = (int)p.M;
      for (int m = 0; m < rows; ++m)
        for (int j = threadIdx.x; j < pieces; j += 32 * kWarps) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.x) + (int64_t)m * pieces + j);
          *reinterpret_cast<uint4*>(x_all + m * x_stride(K) + 16 * j) =
              make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                         __byte_perm(v.y, v.w, 0x7632));
        }
      __syncthreads();
    }

    // ---- multiplying
    float tot[MT][NT][4], acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) tot[i][n][k] = acc[i][n][k] = 0.0f;

    // ldmatrix: lane l names row (l & 7) + 8 (l >> 3 & 1) of block (l >> 4)
    const int lm_row = (lane & 7) + 8 * (lane >> 3 & 1);
    const uint32_t lm_at = ring_at + lm_row * 64;
    const int lm_sw = lm_row >> 1 & 3, lm_block = lane >> 4;
    const uint8_t* x_row[NT];  // this lane's rows of x (columns past the last row are not stored)
    int x_flip[NT];
    int group_row[MT];  // (this lane's row of tile i) * KG, as far as its place within a word goes
    auto aim_use = [&]() {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int64_t row = use.tok.e * p.N + (SWIGLU ? i * cols : 16 * i) + (use.col * wn + nw) * kCols + g;
        group_row[i] = (int)(row & 3) * KG;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int m = min(8 * n + g, use.rows() - 1);
        x_row[n] = XW ? x_all + m * x_stride(K) + 16 * t : ring + MT * kTileBytes + kScaleBytes + m * 256 + 16 * t;
        x_flip[n] = (m & 1) * 64;
      }
    };
    aim_use();

    int slot = 0, c = kw;
    while (true) {
      copy_wait<S - 1>();
      __syncwarp();
      const int blocks = min(4, K / 32 - 4 * c);
      const uint8_t* table = ring + slot * stage_size + MT * kTileBytes;
#pragma unroll
      for (int jj = 0; jj < 4; jj += 2) {
        if (jj >= blocks) break;
        uint32_t words[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
          ldmatrix4(words[i], lm_at + slot * stage_size + i * kTileBytes + 16 * ((jj + lm_block) ^ lm_sw));
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
          const int j = jj + jb;
          if (j >= blocks) break;
          uint32_t b[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (XW) {
              const uint4 v = *reinterpret_cast<const uint4*>(x_row[n] + c * 256 + 64 * j);
              b[n][0] = v.x, b[n][1] = v.y, b[n][2] = v.z, b[n][3] = v.w;
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(x_row[n] + slot * stage_size + (64 * j ^ x_flip[n]));
              b[n][0] = __byte_perm(v.x, v.z, 0x5410);
              b[n][1] = __byte_perm(v.x, v.z, 0x7632);
              b[n][2] = __byte_perm(v.y, v.w, 0x5410);
              b[n][3] = __byte_perm(v.y, v.w, 0x7632);
            }
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            float sl, sh;
            uint32_t zl = kMagic<XT> + 0x80008u, zh = zl;
            {
              // rows g and g + 8 start alike within a word: 8 KG is a multiple of 4
              const int first = group_row[i] + c * kGroups;
              const uint8_t* sp = table + (16 * i + g) * kScaleWords * 4 + 2 * ((first & 1) + j / GB);
              const uint32_t l = *reinterpret_cast<const uint16_t*>(sp);
              const uint32_t h = *reinterpret_cast<const uint16_t*>(sp + 8 * kScaleWords * 4);
              sl = p.scale_dtype == SP24_BF16 ? W4Half<SP24_BF16>::get(l) : W4Half<SP24_F16>::get(l);
              sh = p.scale_dtype == SP24_BF16 ? W4Half<SP24_BF16>::get(h) : W4Half<SP24_F16>::get(h);
              if (ZEROS) {
                const uint8_t* zp = table + kZeroAt + (16 * i + g) * kZeroWords * 4 + (first & 3) + j / GB;
                zl = kMagic<XT> + (zp[0] & 15u) * 0x10001u;
                zh = kMagic<XT> + (zp[8 * kZeroWords * 4] & 15u) * 0x10001u;
              }
            }
            uint32_t lo[4], hi[4];
            expand8<XT>(words[i][2 * jb], zl, lo);
            expand8<XT>(words[i][2 * jb + 1], zh, hi);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t a[4] = {lo[2 * half], hi[2 * half], lo[2 * half + 1], hi[2 * half + 1]};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816<XT>(acc[i][n], a, b[n][2 * half], b[n][2 * half + 1]);
            }
            if ((j + 1) % GB == 0) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  tot[i][n][k] = fmaf(k < 2 ? sl : sh, acc[i][n][k], tot[i][n][k]);
                  acc[i][n][k] = 0.0f;
                }
            }
          }
        }
      }
      __syncwarp();
      fetch(slot);
      slot = slot + 1 == S ? 0 : slot + 1;
      c += wk;
      if (c < chunks) continue;

      // ---- the item is done: partial[warp][tile][token][row]
      const int rows = use.rows();
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int m = 8 * n + 2 * t + (k & 1);
            if (m < rows) partial[((warp * MT + i) * kTok + m) * 16 + g + 8 * (k >> 1)] = tot[i][n][k];
            tot[i][n][k] = 0.0f;
          }
      __syncthreads();
      constexpr int kOutTiles = SWIGLU ? 1 : MT;
      for (int o = threadIdx.x; o < rows * wn * kOutTiles * 16; o += 32 * kWarps) {
        const int r = o & 15, m = (o >> 4) / (kOutTiles * wn), tile = (o >> 4) - m * (kOutTiles * wn);
        const int i = tile & (kOutTiles - 1), w = tile / kOutTiles;
        const int64_t col = use.col * (kCols * wn) + tile * 16 + r;
        if (col >= cols) continue;
        float v = 0.0f, up = 0.0f;
        for (int k = 0; k < wk; ++k) {
          v += partial[(((w * wk + k) * MT + i) * kTok + m) * 16 + r];
          if (SWIGLU) up += partial[(((w * wk + k) * MT + 1) * kTok + m) * 16 + r];
        }
        if (SWIGLU) v = v / (1.0f + expf(-v)) * up;
        const int64_t at = (use.tok.m0 + m) * cols + col;
        if (p.y_f32)
          reinterpret_cast<float*>(p.y)[at] = v;
        else
          reinterpret_cast<uint16_t*>(p.y)[at] = (uint16_t)W4Half<XT>::put(v);
      }
      partial = partial == reinterpret_cast<float*>(smem) ? partial + kPartial : reinterpret_cast<float*>(smem);
      c = kw;
      use.advance(p, col_tiles);
      if (use.left <= 0) break;
      aim_use();
    }
    copy_wait<0>();
  }
};

template <int XT, int NT, int MT, int S, bool SWIGLU, bool XW, bool ZEROS, int GB>
__global__ void __launch_bounds__(32 * kWarps, 2) gemv_w4_kernel(const __grid_constant__ GemvW4 p) {
  extern __shared__ __align__(128) uint8_t smem[];
  GemvKernel<XT, NT, MT, S, SWIGLU, XW, ZEROS, GB>::run(p, smem);
}

template <int XT, int NT, int MT, int S, bool SWIGLU, bool XW, bool ZEROS, int GB>
int launch_gemv(const GemvW4& p, cudaStream_t s) {
  using Kern = GemvKernel<XT, NT, MT, S, SWIGLU, XW, ZEROS, GB>;
  auto kernel = gemv_w4_kernel<XT, NT, MT, S, SWIGLU, XW, ZEROS, GB>;
  const int64_t bytes = Kern::smem_bytes(p);
  // what one SM holds of this kernel: the register limit is asked for once per device
  static int by_regs[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SP24_ERR_CUDA;
  if (!by_regs[dev]) {
    cudaFuncAttributes a;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448) != cudaSuccess ||
        cudaFuncGetAttributes(&a, kernel) != cudaSuccess)
      return SP24_ERR_CUDA;
    by_regs[dev] = 65536 / ((a.numRegs + 7) / 8 * 8 * 32 * kWarps);
  }
  const int64_t by_smem = 233472 / (bytes + 1024);
  const int64_t per_sm = by_smem < by_regs[dev] ? by_smem : by_regs[dev];
  const int64_t cols = SWIGLU ? p.N / 2 : p.N, per_cta = (int64_t)Kern::kCols * (kWarps / p.wk);
  const int64_t col_tiles = (cols + per_cta - 1) / per_cta;
  // with experts: the sum of ceil(rows / kTok) is at most this
  const int64_t tok_tiles = (p.M + Kern::kTok - 1) / Kern::kTok + (p.offsets ? (p.E < p.M ? p.E : p.M) : 0);
  const int64_t room = (per_sm < 1 ? 1 : per_sm) * sm_count(), items = col_tiles * tok_tiles;
  kernel<<<(unsigned)(items < room ? items : room), 32 * kWarps, (size_t)bytes, s>>>(p);
  return launch_status();
}

template <int XT, int NT, int MT, int S, bool SWIGLU, bool XW>
int by_group(const GemvW4& p, cudaStream_t s) {
  if (p.zeros) {
    if (p.group == 128) return launch_gemv<XT, NT, MT, S, SWIGLU, XW, true, 4>(p, s);
    if (p.group == 64) return launch_gemv<XT, NT, MT, S, SWIGLU, XW, true, 2>(p, s);
    return launch_gemv<XT, NT, MT, S, SWIGLU, XW, true, 1>(p, s);
  }
  if (p.group == 128) return launch_gemv<XT, NT, MT, S, SWIGLU, XW, false, 4>(p, s);
  if (p.group == 64) return launch_gemv<XT, NT, MT, S, SWIGLU, XW, false, 2>(p, s);
  return launch_gemv<XT, NT, MT, S, SWIGLU, XW, false, 1>(p, s);
}

template <int XT>
int gemv_by_shape(GemvW4 p, cudaStream_t s) {
  const int64_t chunks = (p.K + kChunk - 1) / kChunk;
  p.wk = chunks >= 8 ? 8 : chunks >= 4 ? 4 : chunks >= 2 ? 2 : 1;
  // sixteen rows of x per tile only where eight would leave a second tile per matrix
  const bool wide = p.M > 8 * p.E;
  const int tok = wide ? 16 : 8;
  p.x_rows = (int)(p.M < tok ? p.M : tok);
  const bool whole = !p.offsets && p.x_rows * p.K <= 16384;  // at most 32 KB of shared memory for x
  if (p.act == SP24_ACT_SWIGLU) {
    if (wide) return by_group<XT, 2, 2, 2, true, false>(p, s);
    return whole ? by_group<XT, 1, 2, 3, true, true>(p, s) : by_group<XT, 1, 2, 2, true, false>(p, s);
  }
  if (wide) return by_group<XT, 2, 2, 2, false, false>(p, s);
  return whole ? by_group<XT, 1, 1, 6, false, true>(p, s) : by_group<XT, 1, 2, 2, false, false>(p, s);
}

}  // namespace
}  // namespace sp24
