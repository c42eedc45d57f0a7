// Programmatic dependent launch: a kernel is set up while the one before it in the stream
// still runs (a chain of short kernels costs about 1 us less for each).  All kernels
// launched so wait before they touch memory that others write, and no thread exits without
// having waited: "the grid before is complete" then holds for all grids before it.
#pragma once

#include "common.cuh"

namespace sfm {

#ifdef __CUDACC__
// How such a kernel reads what others may have written, inputs included: by plain loads, after the
// wait.  The read-only path (__ldg, or const __restrict__ parameters) is open only to what nobody
// writes while the kernel runs, and it runs from before its wait on: the compiler may move such a
// load above the wait.
template <typename T>
__device__ __forceinline__ T load_late(const T* p) {
  return *p;
}
// Waits until the grid this one depends on has completed and its writes are visible.
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// In the grid depended on, after its own wait: the dependent one may be set up from here on.
// What it reads before its wait may then be anything that this grid does not write.
__device__ __forceinline__ void grid_dependency_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

// Launches a kernel that may be set up while the previous one in the stream still runs, its CTAs
// in clusters of that size.
template <typename... P, typename... A>
cudaError_t launch_dependent_clusters(void (*kernel)(P...), int cluster, unsigned grid, unsigned block, size_t smem,
                                      cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                             A... args) {
  return launch_dependent_clusters(kernel, 1, grid, block, smem, s, args...);
}

}  // namespace sfm
