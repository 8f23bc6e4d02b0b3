// 4-bit integer weights with one scale (and zero point) per group of 32, 64 or 128 entries of a
// row: quantiser, dequantiser, and the products of a few rows with such weights (definitions in
// sp24.h).
#include "sp24_internal.cuh"

namespace sp24 {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

template <int DT>
struct Half16;
template <>
struct Half16<SP24_BF16> {
  static __device__ __forceinline__ float get(uint32_t h) { return __uint_as_float(h << 16); }
  static __device__ __forceinline__ uint32_t put(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
};
template <>
struct Half16<SP24_F16> {
  static __device__ __forceinline__ float get(uint32_t h) { return __half2float(__ushort_as_half((unsigned short)h)); }
  static __device__ __forceinline__ uint32_t put(float v) { return __half_as_ushort(__float2half_rn(v)); }
};

__device__ __forceinline__ float scale16(const uint16_t* s, int64_t i, int dtype) {
  return dtype == SP24_BF16 ? Half16<SP24_BF16>::get(s[i]) : Half16<SP24_F16>::get(s[i]);
}

// ------------------------------------------------------------------ quantise

// Eight entries per thread (one 16-byte load, one code word), G / 8 neighbouring lanes per group.
//
// Why a reciprocal is enough: w and s are 16-bit floats with significands below 2^11, and |w| >= s/2
// where a border matters, so |2w - (2n + 1) s| is 0 or at least s's last place: a quotient w / s that
// is not exactly on a border n + 1/2 is at least 2^-12 away from it.  fma(w, 1/s, 1/2) is within
// 2^-18 of w / s + 1/2 (|w / s| < 32), so with 2^-16 added its floor is that of the exact value, and
// an exact border goes up.
template <int DT>
__global__ void __launch_bounds__(256) quantize_w4_kernel(const uint4* __restrict__ w, int64_t vecs, int group,
                                                          int with_zeros, uint32_t* __restrict__ codes,
                                                          uint16_t* __restrict__ scales, uint8_t* __restrict__ zeros) {
  const int span = group / 8;  // lanes per group: 4, 8 or 16
  for (int64_t base = (int64_t)blockIdx.x * 256; base < vecs; base += (int64_t)gridDim.x * 256) {
    const int64_t i = base + threadIdx.x;
    const uint4 x = i < vecs ? ldg_stream16(w + i) : make_uint4(0, 0, 0, 0);
    const uint32_t word[4] = {x.x, x.y, x.z, x.w};
    float v[8];
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = Half16<DT>::get(word[k] & 0xffffu);
      v[2 * k + 1] = Half16<DT>::get(word[k] >> 16);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      lo = fminf(lo, v[k]);
      hi = fmaxf(hi, v[k]);
    }
    for (int d = span / 2; d; d >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(kFull, lo, d));
      hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, d));
    }
    const float width = with_zeros ? __fdiv_rn(hi - lo, 15.0f) : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
    uint32_t s16 = Half16<DT>::put(width);
    float s = Half16<DT>::get(s16);
    if (!(s >= 0x1p-126f)) s16 = 0, s = 0.0f;
    const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
    constexpr float kHalf = 0.5f + 0x1p-16f;
    float z = 8.0f;
    if (with_zeros) z = s > 0.0f ? fminf(fmaxf(floorf(fmaf(-lo, inv, kHalf)), 0.0f), 15.0f) : 0.0f;
    uint32_t out = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float q = fminf(fmaxf(floorf(fmaf(v[k], inv, kHalf)) + z, 0.0f), 15.0f);
      out |= (uint32_t)(int)q << (4 * k);
    }
    if (i < vecs) {
      codes[i] = out;
      if (threadIdx.x % span == 0) {
        scales[i / span] = (uint16_t)s16;
        if (with_zeros) zeros[i / span] = (uint8_t)(int)z;
      }
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(256) dequantize_w4_kernel(const uint32_t* __restrict__ codes,
                                                            const uint16_t* __restrict__ scales, int scale_dtype,
                                                            const uint8_t* __restrict__ zeros, int64_t vecs, int group,
                                                            void* __restrict__ out) {
  const int span = group / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < vecs; i += (int64_t)gridDim.x * 256) {
    const uint32_t c = codes[i];
    const float s = scale16(scales, i / span, scale_dtype);
    const int z = zeros ? zeros[i / span] & 15 : 8;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = (float)((int)(c >> (4 * k) & 15) - z) * s;
    if (DT == SP24_F32) {
      float4* o = reinterpret_cast<float4*>(out) + 2 * i;
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      constexpr int D = DT == SP24_F32 ? SP24_F16 : DT;
      uint32_t p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = Half16<D>::put(v[2 * k]) | Half16<D>::put(v[2 * k + 1]) << 16;
      reinterpret_cast<uint4*>(out)[i] = make_uint4(p[0], p[1], p[2], p[3]);
    }
  }
}

// ------------------------------------------------------------------ products

struct GemvW4 {
  const void* x;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  const int32_t* offsets;  // grouped: E + 1
  void* y;
  int64_t M, E, N, K;
  int scale_dtype, group, y_f32;
  int wk;      // warps along K (a power of two); the other 8 / wk take further columns
  int x_rows;  // rows of x that shared memory has room for
};

constexpr int kWarps = 8;
constexpr int kChunk = 128;     // entries of K per stage: 64 code bytes of each row
constexpr int kTileBytes = 16 * kChunk / 2;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src));
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

// Tile `tile` of all experts' tiles of `rows` rows: its expert, first row and end (one warp).
// Each lane sums the tiles of a contiguous run of experts; the run that holds the tile is then
// looked through by all lanes.
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ offsets, int64_t E, int64_t M, int64_t tile,
                                          int rows, int64_t& e, int64_t& m0, int64_t& m1) {
  const int lane = threadIdx.x & 31;
  auto tiles_of = [&](int64_t i, int64_t& a, int64_t& b) {
    a = max(0, offsets[i]);
    b = min(M, (int64_t)offsets[i + 1]);
    return b > a ? (b - a + rows - 1) / rows : 0;
  };
  auto scan = [&](int64_t v) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(kFull, v, d);
      if (lane >= d) v += o;
    }
    return v;
  };
  const int64_t per = (E + 31) / 32;
  int64_t mine = 0, a, b;
  for (int64_t i = lane * per; i < min(E, (lane + 1) * per); ++i) mine += tiles_of(i, a, b);
  int64_t upto = scan(mine);
  const unsigned past = __ballot_sync(kFull, upto > tile);
  if (!past) return false;
  const int who = __ffs(past) - 1;
  tile -= __shfl_sync(kFull, upto - mine, who);
  for (int64_t i0 = who * per; i0 < min(E, (who + 1) * per); i0 += 32) {
    const int64_t i = i0 + lane;
    mine = i < min(E, (who + 1) * per) ? tiles_of(i, a, b) : 0;
    upto = scan(mine);
    const unsigned hit = __ballot_sync(kFull, upto > tile);
    if (hit) {
      const int l = __ffs(hit) - 1;
      e = i0 + l;
      const int64_t first = __shfl_sync(kFull, a, l);
      m1 = __shfl_sync(kFull, b, l);
      m0 = first + (tile - __shfl_sync(kFull, upto - mine, l)) * rows;
      return true;
    }
    tile -= __shfl_sync(kFull, upto, 31);
  }
  return false;
}

// y = x W^T for up to 8 NT rows of x and MT tiles of 16 weight rows per warp (with SwiGLU: a gate
// tile and its up tile).  The weight rows are the MMA's M, the rows of x its N.
//
// K is split over wk warps of the CTA in chunks of 128 entries; each warp streams its chunks of
// codes through a ring of S stages of its own with cp.async, so nothing in the loop waits for
// another warp.  An ldmatrix of 16-byte row pieces hands lane (g, t) the eight codes 8t .. 8t + 7 of
// a 32-entry block of rows g and g + 8; the MMA may sum K in any order, so the pairs that expand8
// gives are fed as they come, with x's pairs picked alike.  A group's sum is scaled in fp32; the
// warps' partial sums meet in shared memory in a fixed order.
//
// XW: x stands in shared memory whole, its pairs picked when it is brought there (few rows of x);
// otherwise its chunk travels in the ring and the pairs are picked at each use.
template <int XT, int NT, int MT, int S, bool SWIGLU, bool XW, bool ZEROS, int GB>
__global__ void __launch_bounds__(32 * kWarps) gemv_w4_kernel(const __grid_constant__ GemvW4 p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  constexpr int kTok = 8 * NT;
  int64_t e = 0, m0 = (int64_t)blockIdx.y * kTok, m1 = p.M;
  if (p.offsets && !find_tile(p.offsets, p.E, p.M, blockIdx.y, kTok, e, m0, m1)) return;
  const int rows = (int)min((int64_t)kTok, m1 - m0);

  const int wk = p.wk, wn = kWarps / wk;
  const int kw = warp & (wk - 1), nw = warp / wk;
  constexpr int kCols = SWIGLU ? 16 : 16 * MT;  // output columns per warp
  const int64_t cols = SWIGLU ? p.N / 2 : p.N;
  const int64_t cta_col = (int64_t)blockIdx.x * kCols * wn, col0 = cta_col + nw * kCols;
  // weight row r of this warp's tile i (rows past the end: the last one, computed and not stored)
  auto tile_row = [&](int i, int r) {
    const int64_t c = min(col0 + (SWIGLU ? r : 16 * i + r), cols - 1);
    return e * p.N + (SWIGLU ? i * cols : 0) + c;
  };
  const int K = (int)p.K, KG = K / (32 * GB);
  const int chunks = (K + kChunk - 1) / kChunk;

  constexpr int kGroups = 4 / GB;                       // groups per chunk
  constexpr int kScales = 16 * MT * kGroups;            // of all rows
  constexpr int kPer = (kScales + 31) / 32;             // per lane
  constexpr int kWord = ZEROS ? 8 : 4;                  // the scale, and the zero point beside it
  const int stage_bytes = MT * kTileBytes + (XW ? 0 : p.x_rows * 2 * kChunk);
  const int warp_bytes = S * stage_bytes + 2 * kScales * kWord;
  uint8_t* ring = smem + warp * warp_bytes;
  uint8_t* table = ring + S * stage_bytes;
  uint8_t* x_all = smem + kWarps * warp_bytes;
  const int x_stride = (2 * K + 127) / 128 * 128 + 64;  // two neighbouring rows of x never meet in a bank

  const uint8_t* code_src[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      code_src[i][h] = p.codes + tile_row(i, g + 8 * h) * (p.K / 2) + 16 * t + kw * (kChunk / 2);
  const uint8_t* x_src = reinterpret_cast<const uint8_t*>(p.x) + m0 * p.K * 2;
  const uint32_t ring_at = smem_addr(ring);
  const uint32_t code_dst = ring_at + g * 64 + 16 * (t ^ (g >> 1 & 3));  // rows g and g + 8 swizzle alike

  auto fetch = [&](int c, int slot) {  // chunks in order: the sources move on with each call
    const int k0 = c * kChunk;
    const uint32_t dst = code_dst + slot * stage_bytes;
    if (k0 + 32 * t < K) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) copy16(dst + i * kTileBytes + h * 512, code_src[i][h]);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) code_src[i][h] += wk * (kChunk / 2);
    if (!XW) {  // x: row m's 256 bytes at 256 m, its 16-byte piece j at 16 (j ^ 4 (m & 1))
      const uint32_t xdst = ring_at + slot * stage_bytes + MT * kTileBytes;
      for (int j = lane; j < rows * 16; j += 32) {
        const int m = j >> 4, piece = j & 15;
        if (k0 + 8 * piece < K)
          copy16(xdst + m * 256 + 16 * (piece ^ (m & 1) * 4), x_src + ((int64_t)m * K + k0 + 8 * piece) * 2);
      }
    }
  };

  // scales (and zero points) of a chunk: one chunk ahead in registers, then in a table of two turns
  int64_t scale_at[kPer];
  int scale_group[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = lane + 32 * i, r = s / kGroups;
    scale_group[i] = s < kScales ? kw * kGroups + s % kGroups : KG;
    scale_at[i] = tile_row(r >> 4 & (MT - 1), r & 15) * KG + scale_group[i];
  }
  uint32_t scale_bits[kPer], zero_bits[kPer];
  auto load_scales = [&]() {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      scale_bits[i] = 0;
      zero_bits[i] = 8;
      if (scale_group[i] < KG) {
        scale_bits[i] = p.scales[scale_at[i]];
        if (ZEROS) zero_bits[i] = p.zeros[scale_at[i]];
      }
      scale_group[i] += wk * kGroups;
      scale_at[i] += wk * kGroups;
    }
  };
  auto put_scales = [&](int turn) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = lane + 32 * i;
      if (s >= kScales) break;
      const float v = p.scale_dtype == SP24_BF16 ? Half16<SP24_BF16>::get(scale_bits[i]) : Half16<SP24_F16>::get(scale_bits[i]);
      if (ZEROS)
        reinterpret_cast<uint2*>(table)[turn * kScales + s] =
            make_uint2(__float_as_uint(v), kMagic<XT> + (zero_bits[i] & 15u) * 0x10001u);
      else
        reinterpret_cast<float*>(table)[turn * kScales + s] = v;
    }
  };

#pragma unroll
  for (int s = 0; s < S; ++s) {
    if (kw + s * wk < chunks) fetch(kw + s * wk, s);
    copy_commit();
  }
  load_scales();
  if (XW) {
    const int pieces = K / 8;
    for (int m = 0; m < rows; ++m)
      for (int j = threadIdx.x; j < pieces; j += 32 * kWarps) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(x_src) + (int64_t)m * pieces + j);
        *reinterpret_cast<uint4*>(x_all + m * x_stride + 16 * j) =
            make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                       __byte_perm(v.y, v.w, 0x7632));
      }
    __syncthreads();
  }

  float tot[MT][NT][4];
  float acc[MT][NT][4];
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
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int m = min(8 * n + g, rows - 1);
    x_row[n] = XW ? x_all + m * x_stride + 16 * t : ring + MT * kTileBytes + m * 256 + 16 * t;
    x_flip[n] = (m & 1) * 64;
  }

  int slot = 0, turn = 0;
  for (int c = kw; c < chunks; c += wk) {
    put_scales(turn);
    load_scales();
    copy_wait<S - 1>();
    __syncwarp();
    const int blocks = min(4, K / 32 - 4 * c);
#pragma unroll
    for (int jj = 0; jj < 4; jj += 2) {
      if (jj >= blocks) break;
      uint32_t words[MT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
        ldmatrix4(words[i], lm_at + slot * stage_bytes + i * kTileBytes + 16 * ((jj + lm_block) ^ lm_sw));
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
            const uint4 v = *reinterpret_cast<const uint4*>(x_row[n] + slot * stage_bytes + (64 * j ^ x_flip[n]));
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
          const int at = turn * kScales + (16 * i + g) * kGroups + j / GB;
          if (ZEROS) {
            const uint2 l = reinterpret_cast<const uint2*>(table)[at], h = reinterpret_cast<const uint2*>(table)[at + 8 * kGroups];
            sl = __uint_as_float(l.x), zl = l.y, sh = __uint_as_float(h.x), zh = h.y;
          } else {
            sl = reinterpret_cast<const float*>(table)[at], sh = reinterpret_cast<const float*>(table)[at + 8 * kGroups];
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
    if (c + S * wk < chunks) fetch(c + S * wk, slot);
    copy_commit();
    slot = slot + 1 == S ? 0 : slot + 1;
    turn ^= 1;
  }
  copy_wait<0>();
  __syncthreads();  // every warp is past its ring: the partial sums take its place

  // partial[warp][tile][token][row]
  float* partial = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        partial[((warp * MT + i) * kTok + 8 * n + 2 * t + (k & 1)) * 16 + g + 8 * (k >> 1)] = tot[i][n][k];
  __syncthreads();
  constexpr int kOutTiles = SWIGLU ? 1 : MT;
  for (int o = threadIdx.x; o < wn * kOutTiles * kTok * 16; o += 32 * kWarps) {
    const int r = o & 15, tile = (o >> 4) % (kOutTiles * wn), m = (o >> 4) / (kOutTiles * wn);
    const int i = tile % kOutTiles, w = tile / kOutTiles;
    const int64_t col = cta_col + tile * 16 + r;
    if (m >= rows || col >= cols) continue;
    float v = 0.0f, up = 0.0f;
    for (int k = 0; k < wk; ++k) {
      v += partial[(((w * wk + k) * MT + i) * kTok + m) * 16 + r];
      if (SWIGLU) up += partial[(((w * wk + k) * MT + 1) * kTok + m) * 16 + r];
    }
    if (SWIGLU) v = v / (1.0f + expf(-v)) * up;
    const int64_t at = (m0 + m) * cols + col;
    if (p.y_f32)
      reinterpret_cast<float*>(p.y)[at] = v;
    else
      reinterpret_cast<uint16_t*>(p.y)[at] = (uint16_t)Half16<XT>::put(v);
  }
}

template <int XT, int NT, int MT, int S, bool SWIGLU, bool XW, bool ZEROS, int GB>
int launch_gemv(const GemvW4& p, int64_t tiles, cudaStream_t s) {
  auto kernel = gemv_w4_kernel<XT, NT, MT, S, SWIGLU, XW, ZEROS, GB>;
  const int wn = kWarps / p.wk;
  const int64_t cols = SWIGLU ? p.N / 2 : p.N, per_cta = (int64_t)(SWIGLU ? 16 : 16 * MT) * wn;
  const int64_t stage = MT * kTileBytes + (XW ? 0 : p.x_rows * 2 * kChunk);
  const int64_t ring = kWarps * (S * stage + 2 * 16 * MT * (4 / GB) * (ZEROS ? 8 : 4));
  const int64_t bytes = ring + (XW ? p.x_rows * ((2 * p.K + 127) / 128 * 128 + 64) : 0);
  static bool raised[64];  // the attribute holds per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SP24_ERR_CUDA;
  if (dev < 0 || dev >= 64 || !raised[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448) != cudaSuccess)
      return SP24_ERR_CUDA;
    if (dev >= 0 && dev < 64) raised[dev] = true;
  }
  kernel<<<dim3((unsigned)((cols + per_cta - 1) / per_cta), (unsigned)tiles), 32 * kWarps, (size_t)bytes, s>>>(p);
  return launch_status();
}

template <int XT, int NT, int MT, int S, bool SWIGLU, bool XW>
int by_group(const GemvW4& p, int64_t tiles, cudaStream_t s) {
  if (p.zeros) {
    if (p.group == 128) return launch_gemv<XT, NT, MT, S, SWIGLU, XW, true, 4>(p, tiles, s);
    if (p.group == 64) return launch_gemv<XT, NT, MT, S, SWIGLU, XW, true, 2>(p, tiles, s);
    return launch_gemv<XT, NT, MT, S, SWIGLU, XW, true, 1>(p, tiles, s);
  }
  if (p.group == 128) return launch_gemv<XT, NT, MT, S, SWIGLU, XW, false, 4>(p, tiles, s);
  if (p.group == 64) return launch_gemv<XT, NT, MT, S, SWIGLU, XW, false, 2>(p, tiles, s);
  return launch_gemv<XT, NT, MT, S, SWIGLU, XW, false, 1>(p, tiles, s);
}

template <int XT>
int by_shape(GemvW4& p, bool grouped, int act, cudaStream_t s) {
  const int64_t chunks = (p.K + kChunk - 1) / kChunk;
  p.wk = chunks >= 8 ? 8 : chunks >= 4 ? 4 : chunks >= 2 ? 2 : 1;
  // sixteen rows of x per tile only where eight would leave a second tile per matrix
  const bool wide = grouped ? p.M > 8 * p.E : p.M > 8;
  const int tok = wide ? 16 : 8;
  p.x_rows = (int)(p.M < tok ? p.M : tok);
  // grouped: the sum over experts of ceil(rows / tok) is at most this
  const int64_t tiles = (p.M + tok - 1) / tok + (grouped ? (p.E < p.M ? p.E : p.M) : 0);
  if (tiles > 65535) return SP24_ERR_UNSUPPORTED;
  const bool whole = p.x_rows * p.K <= 16384;  // at most 32 KB of shared memory for x
  if (act == SP24_ACT_SWIGLU) {
    if (wide) return by_group<XT, 2, 2, 2, true, false>(p, tiles, s);
    return whole ? by_group<XT, 1, 2, 2, true, true>(p, tiles, s) : by_group<XT, 1, 2, 2, true, false>(p, tiles, s);
  }
  if (wide) return by_group<XT, 2, 2, 2, false, false>(p, tiles, s);
  return whole ? by_group<XT, 1, 1, 4, false, true>(p, tiles, s) : by_group<XT, 1, 2, 2, false, false>(p, tiles, s);
}

bool is16(int d) { return d == SP24_F16 || d == SP24_BF16; }

int check_w4(int64_t rows, int64_t K, int group) {
  if (group != 32 && group != 64 && group != 128) return SP24_ERR_UNSUPPORTED;
  if (rows < 0 || K < 0 || K % group) return SP24_ERR_SHAPE;
  return SP24_OK;
}

int gemv(const void* x, int x_dtype, const sp24_w4_operand* w, const int32_t* offsets, bool grouped, int64_t M,
         int64_t E, int64_t N, int64_t K, int act, void* y, int y_dtype, cudaStream_t s) {
  if (!w) return SP24_ERR_INVALID_ARG;
  if (act != SP24_ACT_NONE && act != SP24_ACT_SWIGLU) return SP24_ERR_INVALID_ARG;
  if (!is16(x_dtype) || !is16(w->scale_dtype) || (y_dtype != SP24_F32 && y_dtype != x_dtype)) return SP24_ERR_DTYPE;
  const int st = check_w4(N, K, w->group);
  if (st) return st;
  if (M < 0 || E < 1 || (act == SP24_ACT_SWIGLU && N % 2)) return SP24_ERR_SHAPE;
  if (M > INT32_MAX || E > INT32_MAX || N > INT32_MAX || K > INT32_MAX / 2) return SP24_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return SP24_OK;
  const int64_t cols = act == SP24_ACT_SWIGLU ? N / 2 : N;
  const int yb = elem_bytes(y_dtype);
  if (!y || (grouped && !offsets)) return SP24_ERR_INVALID_ARG;
  if (!aligned(y, yb) || !aligned(offsets, 4)) return SP24_ERR_ALIGN;
  if (K == 0) return cudaMemsetAsync(y, 0, (size_t)(M * cols * yb), s) == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
  if (!x || !w->codes || !w->scales) return SP24_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w->codes, 16) || !aligned(w->scales, 2)) return SP24_ERR_ALIGN;
  GemvW4 p{x, w->codes, reinterpret_cast<const uint16_t*>(w->scales), w->zeros, grouped ? offsets : nullptr, y,
           M, E, N, K, w->scale_dtype, w->group, y_dtype == SP24_F32, 0, 0};
  return x_dtype == SP24_BF16 ? by_shape<SP24_BF16>(p, grouped, act, s) : by_shape<SP24_F16>(p, grouped, act, s);
}

unsigned stream_ctas(int64_t vecs) {
  const int64_t need = (vecs + 255) / 256, cap = (int64_t)sm_count() * 8;
  return (unsigned)(need < cap ? need : cap);
}

}  // namespace
}  // namespace sp24

using namespace sp24;

extern "C" int sp24_quantize_w4(const void* w, int dtype, int64_t rows, int64_t K, int group, int with_zeros,
                                uint8_t* codes, void* scales, uint8_t* zeros, void* stream) {
  if (!is16(dtype)) return SP24_ERR_DTYPE;
  const int st = check_w4(rows, K, group);
  if (st) return st;
  if (!zeros != !with_zeros) return SP24_ERR_INVALID_ARG;
  if (rows == 0 || K == 0) return SP24_OK;
  if (!w || !codes || !scales) return SP24_ERR_INVALID_ARG;
  if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales, 2)) return SP24_ERR_ALIGN;
  const int64_t vecs = rows * (K / 8);
  if (dtype == SP24_BF16)
    quantize_w4_kernel<SP24_BF16><<<stream_ctas(vecs), 256, 0, as_stream(stream)>>>(
        reinterpret_cast<const uint4*>(w), vecs, group, with_zeros, reinterpret_cast<uint32_t*>(codes),
        reinterpret_cast<uint16_t*>(scales), zeros);
  else
    quantize_w4_kernel<SP24_F16><<<stream_ctas(vecs), 256, 0, as_stream(stream)>>>(
        reinterpret_cast<const uint4*>(w), vecs, group, with_zeros, reinterpret_cast<uint32_t*>(codes),
        reinterpret_cast<uint16_t*>(scales), zeros);
  return launch_status();
}

extern "C" int sp24_dequantize_w4(const sp24_w4_operand* w, int64_t rows, int64_t K, int out_dtype, void* out,
                                  void* stream) {
  if (!w) return SP24_ERR_INVALID_ARG;
  if (!is16(w->scale_dtype) || !elem_bytes(out_dtype)) return SP24_ERR_DTYPE;
  const int st = check_w4(rows, K, w->group);
  if (st) return st;
  if (rows == 0 || K == 0) return SP24_OK;
  if (!w->codes || !w->scales || !out) return SP24_ERR_INVALID_ARG;
  if (!aligned(w->codes, 16) || !aligned(w->scales, 2) || !aligned(out, 16)) return SP24_ERR_ALIGN;
  const int64_t vecs = rows * (K / 8);
  const unsigned ctas = stream_ctas(vecs);
  const uint32_t* c = reinterpret_cast<const uint32_t*>(w->codes);
  const uint16_t* sc = reinterpret_cast<const uint16_t*>(w->scales);
  cudaStream_t s = as_stream(stream);
  if (out_dtype == SP24_F32)
    dequantize_w4_kernel<SP24_F32><<<ctas, 256, 0, s>>>(c, sc, w->scale_dtype, w->zeros, vecs, w->group, out);
  else if (out_dtype == SP24_BF16)
    dequantize_w4_kernel<SP24_BF16><<<ctas, 256, 0, s>>>(c, sc, w->scale_dtype, w->zeros, vecs, w->group, out);
  else
    dequantize_w4_kernel<SP24_F16><<<ctas, 256, 0, s>>>(c, sc, w->scale_dtype, w->zeros, vecs, w->group, out);
  return launch_status();
}

extern "C" int sp24_gemv_w4(const void* x, int x_dtype, const sp24_w4_operand* w, int64_t M, int64_t N, int64_t K,
                            int act, void* y, int y_dtype, void* stream) {
  return gemv(x, x_dtype, w, nullptr, false, M, 1, N, K, act, y, y_dtype, as_stream(stream));
}

extern "C" int sp24_gemv_w4_grouped(const void* x, int x_dtype, const sp24_w4_operand* w, const int32_t* offsets,
                                    int64_t R, int64_t E, int64_t N, int64_t K, int act, void* y, int y_dtype,
                                    void* stream) {
  return gemv(x, x_dtype, w, offsets, true, R, E, N, K, act, y, y_dtype, as_stream(stream));
}
