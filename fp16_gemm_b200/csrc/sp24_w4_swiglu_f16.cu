// Products of f16 rows with 4-bit group weights, gate and up joined by SwiGLU.
#include "sp24_w4_gemv.cuh"

int sp24::gemv_w4_swiglu_f16(const GemvW4& p, cudaStream_t s) { return gemv_w4_swiglu<SP24_F16>(p, s); }
