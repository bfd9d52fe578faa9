// Programmatic dependent launch: a kernel of a chain may be scheduled, and run
// its prologue, while the launch before it in the stream is still finishing.
// It must not read (or overwrite) what that launch writes before
// wait_for_previous_launch returns, which is when that launch has completed
// and its writes are visible.
// Such data is not read through the read-only path (__ldg, const __restrict__
// parameters), whose loads may move up past the wait. Every block waits, so a
// launch's end is also the end of those before it.
#pragma once

#include <cuda_runtime.h>

namespace moe {

__device__ __forceinline__ void wait_for_previous_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// For a launch that the one before it let start after its own wait: what came
// before that one is done, and its writes are seen from here on (TMA too).
__device__ __forceinline__ void fence_previous_results() {
  __threadfence();
  asm volatile("fence.proxy.async;" ::: "memory");
}
// Lets the next launch of the chain be scheduled once every block is here.
__device__ __forceinline__ void allow_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// overlap: as a dependent of the launch before it; cluster: CTAs per cluster.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), int grid, int threads, size_t smem, cudaStream_t s, bool overlap,
                             int cluster, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (overlap) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace moe
