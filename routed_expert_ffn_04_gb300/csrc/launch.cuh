// Programmatic dependent launch: a kernel of a chain may be scheduled, and run
// its prologue, while the launch before it in the stream is still finishing.
// It reads and overwrites nothing of an earlier launch before
// wait_for_previous_launch returns, which is when the launch before has
// completed and what it and its predecessors wrote is visible: the wait alone
// promises that, even for data of launches that have long ended.
// Such data is not read through the read-only path (__ldg, const __restrict__
// parameters), whose loads may move up past the wait. Every block waits, so a
// launch's end is also the end of those before it.
//
// What was complete before the launch before began can be had earlier: that
// launch, once it has waited, releases a word in global memory (publish), and
// a thread that acquires it (published) sees all that the publisher saw. A
// launch that does not find its call's number in the word waits as above, so
// nothing rests on when it looks. No two calls have one number, but a replayed
// graph passes its own again: a chain clears its words, in its last launch or,
// for those that are published later, in its first.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace moe {

__device__ __forceinline__ void wait_for_previous_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void publish(uint64_t* word, uint64_t call) {
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(word), "l"(call) : "memory");
}
__device__ __forceinline__ bool published(const uint64_t* word, uint64_t call) {
  uint64_t v;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(word) : "memory");
  return v == call;
}
// By all threads of a block, before its first use of global memory: returns when
// what the word's publisher saw is visible to them, to TMA too. `flag`: a word of
// shared memory. A block that does not find the call waits for the launch before.
__device__ __forceinline__ void wait_until_published(const uint64_t* word, uint64_t call, volatile int* flag) {
  if (threadIdx.x == 0) *flag = published(word, call) ? 1 : 0;
  __syncthreads();
  if (*flag == 0) wait_for_previous_launch();
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
