// A kernel that is launched while the one before it on the stream still runs: its CTAs
// take their places as the other's leave theirs, and wait there until the other has
// ended and its results are visible. What this saves is the way from one kernel's end
// to the next one's first instruction.
#pragma once

#include <cuda_runtime.h>

namespace fljsd {

// In the kernel launched so, before it touches memory.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// In the kernel before it: the next may be launched from here on. (It never takes the
// place of a CTA of this one: all of them have started by then.)
__device__ __forceinline__ void let_next_launch() {
  asm volatile("griddepcontrol.launch_dependents;");
}

// Only behind a kernel of this library that was launched in the same call: what a
// foreign one lets run past it is not known here.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st,
                             const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace fljsd
