// Programmatic dependent launch: a kernel is set up while the one before it in the stream
// still runs.
#pragma once

#include "common.cuh"

namespace sfm {

#ifdef __CUDACC__
// Waits until the grid this one depends on has
// completed and its writes are visible.  Every thread of a dependent kernel calls it
// before it exits and before it touches anything that grid writes (or whatever came
// before that grid in the stream: that grid itself starts only when that is done).
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// In the grid depended on: the dependent one may be set up from here on (it still waits).
__device__ __forceinline__ void grid_dependency_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

// Launches a kernel that may be set up while the previous one in the stream still runs.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem,
                             cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace sfm
