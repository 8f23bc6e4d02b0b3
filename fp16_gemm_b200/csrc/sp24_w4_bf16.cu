// Products of bf16 rows with 4-bit group weights.
#include "sp24_w4_gemv.cuh"

int sp24::gemv_w4_bf16(const GemvW4& p, cudaStream_t s) { return gemv_w4_plain<SP24_BF16>(p, s); }
