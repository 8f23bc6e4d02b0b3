// Programmatic dependent launch: the kernels that are launched with launch_after start while their
// predecessor in the stream is still ending, so that a launch's latency and a kernel's set-up are
// hidden behind it.  Such a kernel calls begin() in every thread, once, before it touches global memory:
// it waits, in hardware, until its predecessor has ended and its writes are visible, and then lets its own
// successor start (whose predecessor's predecessor has ended then).
//
// What such a kernel reads may be written while it already runs, and what it writes may still be read.
// So no load takes the read-only path (__ldg, ld.global.nc: defined for data that nobody writes while the
// kernel runs), and no pointer is __restrict__: the compiler may choose that path for one that is only
// read, and need not keep accesses through any of them behind begin().
#pragma once

#include "sp24_internal.cuh"

namespace sp24 {

__device__ __forceinline__ void begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Sixteen bytes that are read once: they do not displace others in L1.
__device__ __forceinline__ uint4 load_stream16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
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
