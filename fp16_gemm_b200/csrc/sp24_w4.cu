// 4-bit integer weights with one scale (and zero point) per group of 32, 64 or 128 entries of a
// row: quantiser, dequantiser, and the products of a few rows with such weights (definitions in
// sp24.h).
#include "sp24_w4.cuh"

namespace sp24 {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ float scale16(const uint16_t* s, int64_t i, int dtype) {
  return dtype == SP24_BF16 ? W4Half<SP24_BF16>::get(s[i]) : W4Half<SP24_F16>::get(s[i]);
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
      v[2 * k] = W4Half<DT>::get(word[k] & 0xffffu);
      v[2 * k + 1] = W4Half<DT>::get(word[k] >> 16);
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
    uint32_t s16 = W4Half<DT>::put(width);
    float s = W4Half<DT>::get(s16);
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
      for (int k = 0; k < 4; ++k) p[k] = W4Half<D>::put(v[2 * k]) | W4Half<D>::put(v[2 * k + 1]) << 16;
      reinterpret_cast<uint4*>(out)[i] = make_uint4(p[0], p[1], p[2], p[3]);
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
  if (M > INT32_MAX || E > INT32_MAX || N > INT32_MAX || K > (1 << 24)) return SP24_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return SP24_OK;
  const int64_t cols = act == SP24_ACT_SWIGLU ? N / 2 : N;
  const int yb = elem_bytes(y_dtype);
  if (!y || (grouped && !offsets)) return SP24_ERR_INVALID_ARG;
  if (!aligned(y, yb) || !aligned(offsets, 4)) return SP24_ERR_ALIGN;
  if (K == 0) return cudaMemsetAsync(y, 0, (size_t)(M * cols * yb), s) == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
  if (!x || !w->codes || !w->scales) return SP24_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w->codes, 16) || !aligned(w->scales, 4) || !aligned(w->zeros, 4)) return SP24_ERR_ALIGN;
  const GemvW4 p{x, w->codes, reinterpret_cast<const uint16_t*>(w->scales), w->zeros, grouped ? offsets : nullptr, y,
                 M, E, N, K, w->scale_dtype, w->group, act, y_dtype == SP24_F32, 0};
  return x_dtype == SP24_BF16 ? gemv_w4_bf16(p, s) : gemv_w4_f16(p, s);
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
  if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(zeros, 4)) return SP24_ERR_ALIGN;
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
  if (!aligned(w->codes, 16) || !aligned(w->scales, 4) || !aligned(w->zeros, 4) || !aligned(out, 16)) return SP24_ERR_ALIGN;
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
