// 4-bit integer weights with one scale (and zero point) per group of 32, 64 or 128 entries of a
// row: quantiser, dequantiser, and the products of a few rows with such weights (definitions in
// sp24.h).
#include "sp24_launch.cuh"
#include "sp24_w4.cuh"

namespace sp24 {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ------------------------------------------------------------------ quantise

template <int DT>
struct Pair16;
template <>
struct Pair16<SP24_BF16> {
  using T = __nv_bfloat162;
  static constexpr uint32_t kMagic = 0x43004300u;  // 2^7: its last place is 1
};
template <>
struct Pair16<SP24_F16> {
  using T = __half2;
  static constexpr uint32_t kMagic = 0x64006400u;  // 2^10
};
template <int DT>
__device__ __forceinline__ typename Pair16<DT>::T as_pair(uint32_t w) {
  return reinterpret_cast<const typename Pair16<DT>::T&>(w);
}
template <typename T>
__device__ __forceinline__ uint32_t pair_bits(T v) {
  return reinterpret_cast<const uint32_t&>(v);
}

// G / 16 neighbouring lanes per group, sixteen entries each: two 16-byte loads, two code words.
//
// Why a reciprocal is enough: w and s are 16-bit floats with significands below 2^11, and |w| >= s/2
// where a border matters, so |2w - (2n + 1) s| is 0 or at least s's last place: a quotient w / s that
// is not exactly on a border n + 1/2 is at least 2^-12 away from it.  The code is taken as the
// nearest integer to 15 clamp(w / (15 s) + (z + 2^-16) / 15, 0, 1), which is within 2^-17 of
// clamp(w / s + z + 2^-16, 0, 15): so it is that of the exact value, and an exact border goes up.
//
// Bound by instruction issue before HBM if done plainly (74 us for [12288, 5120] bf16, whose bytes take 24
// at the copy rate; 28 us as it is, 31 with zero points), so the arithmetic is cut to four
// instructions an entry: unpacking, one saturating fma (the clamp is its saturation), one fma that
// adds 1.5 * 2^23 (whose last place is 1, which rounds to the integer), and one integer
// multiply-add that joins the codes with the constant's bits still in them; their sum is
// subtracted from the word at the end.  A scale above 2^100, whose 1 / (15 s) may be subnormal,
// first has w and itself divided by 2^64.
template <int DT, int G, bool ZEROS>
__global__ void __launch_bounds__(256) quantize_w4_kernel(const uint4* w, int64_t groups,
                                                          uint32_t* codes, uint16_t* scales,
                                                          uint8_t* zeros) {
  constexpr int L = G / 16;
  using P = typename Pair16<DT>::T;
  const int lane = threadIdx.x % L;
  const int64_t step = (int64_t)gridDim.x * (256 / L);
  begin();
  // every lane of a group is in range together; those of other groups in the warp may not be
  for (int64_t group = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L; group < (groups + 31) / 32 * 32; group += step) {
    const bool live = group < groups;
    const int64_t at = group * (2 * L) + lane;
    uint4 x[2] = {};
    if (live) {
      x[0] = load_stream16(w + at);
      x[1] = load_stream16(w + at + L);
    }
    const uint32_t word[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    float lo = 0.0f, hi = 0.0f;  // symmetric: hi is the largest magnitude
    if (ZEROS) {
      P a = as_pair<DT>(word[0]), b = a;
#pragma unroll
      for (int k = 1; k < 8; ++k) {
        a = __hmax2(a, as_pair<DT>(word[k]));
        b = __hmin2(b, as_pair<DT>(word[k]));
      }
#pragma unroll
      for (int d = 1; d < L; d <<= 1) {
        a = __hmax2(a, as_pair<DT>(__shfl_xor_sync(kFull, pair_bits(a), d)));
        b = __hmin2(b, as_pair<DT>(__shfl_xor_sync(kFull, pair_bits(b), d)));
      }
      const uint32_t ab = pair_bits(a), bb = pair_bits(b);
      hi = fmaxf(0.0f, fmaxf(W4Half<DT>::get(ab & 0xffffu), W4Half<DT>::get(ab >> 16)));
      lo = fminf(0.0f, fminf(W4Half<DT>::get(bb & 0xffffu), W4Half<DT>::get(bb >> 16)));
    } else {
      P a = __habs2(as_pair<DT>(word[0]));
#pragma unroll
      for (int k = 1; k < 8; ++k) a = __hmax2(a, __habs2(as_pair<DT>(word[k])));
#pragma unroll
      for (int d = 1; d < L; d <<= 1) a = __hmax2(a, as_pair<DT>(__shfl_xor_sync(kFull, pair_bits(a), d)));
      const uint32_t ab = pair_bits(a);
      hi = fmaxf(W4Half<DT>::get(ab & 0xffffu), W4Half<DT>::get(ab >> 16));
    }
    uint32_t s16 = W4Half<DT>::put(ZEROS ? __fdiv_rn(hi - lo, 15.0f) : __fdiv_rn(hi, 7.0f));
    float s = W4Half<DT>::get(s16);
    if (!(s >= 0x1p-126f)) s16 = 0, s = 0.0f;
    const float down = s > 0x1p100f ? 0x1p-64f : 1.0f;
    const float inv = s > 0.0f ? __fdiv_rn(1.0f / 15.0f, s * down) : 0.0f;  // 1 / (15 s) within 2^-23
    constexpr float kMagic = 12582912.0f, kRoom = 0x1p-16f;
    float z = 8.0f;
    // as with the codes: -lo / s, which is at most 15
    if (ZEROS) z = s > 0.0f ? fmaf(__saturatef(fmaf(-lo * down, inv, kRoom / 15.0f)), 15.0f, kMagic) - kMagic : 0.0f;
    const float shift = (z + kRoom) * (1.0f / 15.0f);
    uint32_t out[2];
    float scaled[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      scaled[2 * k] = W4Half<DT>::get(word[k] & 0xffffu);
      scaled[2 * k + 1] = W4Half<DT>::get(word[k] >> 16);
    }
    if (down != 1.0f)
#pragma unroll
      for (int k = 0; k < 16; ++k) scaled[k] *= down;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t sum = 0;
#pragma unroll
      for (int k = 7; k >= 0; --k)
        sum = sum * 16 + __float_as_uint(fmaf(__saturatef(fmaf(scaled[8 * h + k], inv, shift)), 15.0f, kMagic));
      out[h] = sum - 0x4b400000u * 0x11111111u;
    }
    if (live) {
      codes[at] = out[0];
      codes[at + L] = out[1];
      if (lane == 0) {
        scales[group] = (uint16_t)s16;
        if (ZEROS) zeros[group] = (uint8_t)(int)z;
      }
    }
  }
}

// Eight codes per thread and turn, four turns in flight.  Where the output has the scales' type, q - z
// (exact) times s is one multiplication in that type, which rounds once: [12288, 5120] to bf16 takes 26 us
// (24 at the copy rate), against 44 with conversions to fp32 and back.
template <int DT, int ST>
__global__ void __launch_bounds__(256) dequantize_w4_kernel(const uint32_t* codes,
                                                            const uint16_t* scales,
                                                            const uint8_t* zeros, int64_t vecs,
                                                            int span_log, void* out) {
  constexpr int kTurns = 4;
  begin();
  for (int64_t base = (int64_t)blockIdx.x * (256 * kTurns) + threadIdx.x; base < vecs;
       base += (int64_t)gridDim.x * (256 * kTurns)) {
    uint32_t c[kTurns], s16[kTurns], z[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
      const int64_t i = min(base + 256 * k, vecs - 1);
      c[k] = __ldcs(codes + i);
      s16[k] = scales[i >> span_log];
      z[k] = zeros ? zeros[i >> span_log] & 15u : 8u;
    }
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
      const int64_t i = base + 256 * k;
      if (i >= vecs) break;
      if constexpr (DT == ST) {
        using P = typename Pair16<DT>::T;
        const P zero = as_pair<DT>(Pair16<DT>::kMagic + z[k] * 0x10001u), scale = as_pair<DT>(s16[k] * 0x10001u);
        uint32_t v[4];  // entries (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = pair_bits(__hmul2(__hsub2(as_pair<DT>((c[k] >> (4 * j) & 0x000f000fu) | Pair16<DT>::kMagic), zero), scale));
        __stcs(reinterpret_cast<uint4*>(out) + i,
               make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                          __byte_perm(v[2], v[3], 0x7632)));
      } else {
        const float s = W4Half<ST>::get(s16[k]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = (__uint_as_float((c[k] >> (4 * j) & 15u) | 0x4b000000u) - (8388608.0f + (float)z[k])) * s;
        if constexpr (DT == SP24_F32) {
          float4* o = reinterpret_cast<float4*>(out) + 2 * i;
          __stcs(o, make_float4(v[0], v[1], v[2], v[3]));
          __stcs(o + 1, make_float4(v[4], v[5], v[6], v[7]));
        } else {
          uint32_t p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = W4Half<DT>::put(v[2 * j]) | W4Half<DT>::put(v[2 * j + 1]) << 16;
          __stcs(reinterpret_cast<uint4*>(out) + i, make_uint4(p[0], p[1], p[2], p[3]));
        }
      }
    }
  }
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
  if (M > INT32_MAX || E > (1 << 20) || N > INT32_MAX || K > (1 << 24)) return SP24_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return SP24_OK;
  const int64_t cols = act == SP24_ACT_SWIGLU ? N / 2 : N;
  const int yb = elem_bytes(y_dtype);
  if (!y || (grouped && !offsets)) return SP24_ERR_INVALID_ARG;
  if (!aligned(y, yb) || !aligned(offsets, 4)) return SP24_ERR_ALIGN;
  // with experts the kernel runs for K == 0 too (it reads offsets alone): only their rows are cleared
  if (K == 0 && !grouped) return cudaMemsetAsync(y, 0, (size_t)(M * cols * yb), s) == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
  if (K && (!x || !w->codes || !w->scales)) return SP24_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w->codes, 16) || !aligned(w->scales, 16) || !aligned(w->zeros, 16)) return SP24_ERR_ALIGN;
  const GemvW4 p{x, w->codes, reinterpret_cast<const uint16_t*>(w->scales), w->zeros, grouped ? offsets : nullptr, y,
                 M, E, N, K, (int16_t)w->scale_dtype, (int16_t)w->group, y_dtype == SP24_F32, 1, 0};
  if (act == SP24_ACT_SWIGLU) return x_dtype == SP24_BF16 ? gemv_w4_swiglu_bf16(p, s) : gemv_w4_swiglu_f16(p, s);
  return x_dtype == SP24_BF16 ? gemv_w4_bf16(p, s) : gemv_w4_f16(p, s);
}

unsigned stream_ctas(int64_t need) {
  const int64_t cap = (int64_t)sm_count() * 32;
  return (unsigned)(need < cap ? need : cap);
}

template <int DT, int G>
int quantize(const void* w, int64_t groups, bool with_zeros, uint8_t* codes, void* scales, uint8_t* zeros,
             cudaStream_t s) {
  const unsigned ctas = stream_ctas((groups * (G / 16) + 255) / 256);
  return launch_after(with_zeros ? quantize_w4_kernel<DT, G, true> : quantize_w4_kernel<DT, G, false>, ctas, 256, 0, s,
                      reinterpret_cast<const uint4*>(w), groups, reinterpret_cast<uint32_t*>(codes),
                      reinterpret_cast<uint16_t*>(scales), zeros);
}

template <int DT>
int quantize_by_group(int group, const void* w, int64_t entries, bool with_zeros, uint8_t* codes, void* scales,
                      uint8_t* zeros, cudaStream_t s) {
  if (group == 128) return quantize<DT, 128>(w, entries / 128, with_zeros, codes, scales, zeros, s);
  if (group == 64) return quantize<DT, 64>(w, entries / 64, with_zeros, codes, scales, zeros, s);
  return quantize<DT, 32>(w, entries / 32, with_zeros, codes, scales, zeros, s);
}

template <int DT>
int dequantize(const sp24_w4_operand* w, int64_t vecs, void* out, cudaStream_t s) {
  const unsigned ctas = stream_ctas((vecs + 1023) / 1024);
  const uint32_t* c = reinterpret_cast<const uint32_t*>(w->codes);
  const uint16_t* sc = reinterpret_cast<const uint16_t*>(w->scales);
  const int span_log = w->group == 128 ? 4 : w->group == 64 ? 3 : 2;
  return launch_after(w->scale_dtype == SP24_BF16 ? dequantize_w4_kernel<DT, SP24_BF16> : dequantize_w4_kernel<DT, SP24_F16>,
                      ctas, 256, 0, s, c, sc, w->zeros, vecs, span_log, out);
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
  if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(zeros, 16)) return SP24_ERR_ALIGN;
  return dtype == SP24_BF16
             ? quantize_by_group<SP24_BF16>(group, w, rows * K, with_zeros, codes, scales, zeros, as_stream(stream))
             : quantize_by_group<SP24_F16>(group, w, rows * K, with_zeros, codes, scales, zeros, as_stream(stream));
}

extern "C" int sp24_dequantize_w4(const sp24_w4_operand* w, int64_t rows, int64_t K, int out_dtype, void* out,
                                  void* stream) {
  if (!w) return SP24_ERR_INVALID_ARG;
  if (!is16(w->scale_dtype) || !elem_bytes(out_dtype)) return SP24_ERR_DTYPE;
  const int st = check_w4(rows, K, w->group);
  if (st) return st;
  if (rows == 0 || K == 0) return SP24_OK;
  if (!w->codes || !w->scales || !out) return SP24_ERR_INVALID_ARG;
  if (!aligned(w->codes, 16) || !aligned(w->scales, 16) || !aligned(w->zeros, 16) || !aligned(out, 16)) return SP24_ERR_ALIGN;
  const int64_t vecs = rows * (K / 8);
  if (out_dtype == SP24_F32) return dequantize<SP24_F32>(w, vecs, out, as_stream(stream));
  if (out_dtype == SP24_BF16) return dequantize<SP24_BF16>(w, vecs, out, as_stream(stream));
  return dequantize<SP24_F16>(w, vecs, out, as_stream(stream));
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
