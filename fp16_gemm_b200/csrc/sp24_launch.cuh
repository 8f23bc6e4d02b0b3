// Programmatic dependent launch: the kernels that are launched with launch_after start while their
// predecessor in the stream is still ending, so that a launch's latency and a kernel's set-up are
// hidden behind it.  Such a kernel calls begin() in every thread before it touches global memory: it waits, in
// hardware, until its predecessor has ended and its writes are visible, and then lets its own successor
// start.  In this order a kernel that has started knows that all before its predecessor has ended, and
// may read what the predecessor alone does not write.
#pragma once

#include "sp24_internal.cuh"

namespace sp24 {

__device__ __forceinline__ void begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
int launch_after(void (*kernel)(P...), unsigned ctas, unsigned threads, size_t shared_bytes, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared_bytes;
  cfg.stream = s;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  count_launch(1);
  if (e == cudaSuccess) return SP24_OK;
  cudaGetLastError();  // the error is reported by the status
  return SP24_ERR_CUDA;
}

}  // namespace sp24
