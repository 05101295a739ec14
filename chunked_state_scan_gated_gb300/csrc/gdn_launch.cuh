// gdn_launch.cuh -- launches that begin as the kernel before them in the stream ends
// (programmatic stream serialization): the next grid's CTAs are placed while the last CTAs of
// the one before run out, and wait on the device for its end.  A kernel launched so calls
// after_previous() before it touches memory; before_next() lets the one behind it start being
// placed once every CTA has called it (or left).  Saves 1 to 3 us per call of a decode step (one
// or two launches), captured or not.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace gdn {

__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void before_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                          cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  if (e != cudaSuccess) cudaGetLastError();  // reported here: not left for the next call
  return e;
}

// Lets the kernel have `bytes` of shared memory, once per device (two threads that both ask do no
// harm).
template <auto kKernel>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < 64 && (done.load() >> dev & 1)) return e;
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) cudaGetLastError();
  else if (dev < 64) done.fetch_or(1ull << dev);
  return e;
}

}  // namespace gdn
