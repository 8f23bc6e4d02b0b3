// Products of a few rows with 4-bit group weights (sp24_gemv_w4, sp24_gemv_w4_grouped): the kernel
// and its launch for one type of x.  sp24_w4.cu checks the arguments.
#pragma once

#include "sp24_internal.cuh"

namespace sp24 {

template <int DT>
struct W4Half;
template <>
struct W4Half<SP24_BF16> {
  static __device__ __forceinline__ float get(uint32_t h) { return __uint_as_float(h << 16); }
  static __device__ __forceinline__ uint32_t put(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
};
template <>
struct W4Half<SP24_F16> {
  static __device__ __forceinline__ float get(uint32_t h) { return __half2float(__ushort_as_half((unsigned short)h)); }
  static __device__ __forceinline__ uint32_t put(float v) { return __half_as_ushort(__float2half_rn(v)); }
};

// The kernel's parameter block.  Its size shows in a call's time: [5120, 5120] takes 8.3 us a call with 96
// bytes and 8.8 with 104.
struct GemvW4 {
  const void* x;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  const int32_t* offsets;  // grouped: E + 1
  void* y;
  int64_t M, E, N, K;
  int16_t scale_dtype, group, y_f32;
  int16_t share;   // set by the launch: the teams of a CTA that take an item's K together, all or one
  int tile_bound;  // set by the launch, with experts: the most row tiles that ascending offsets give
};
static_assert(sizeof(GemvW4) == 96);

int gemv_w4_bf16(const GemvW4& p, cudaStream_t s);
int gemv_w4_f16(const GemvW4& p, cudaStream_t s);
int gemv_w4_swiglu_bf16(const GemvW4& p, cudaStream_t s);
int gemv_w4_swiglu_f16(const GemvW4& p, cudaStream_t s);

}  // namespace sp24
