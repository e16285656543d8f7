// follow.cuh -- kernels that may be put on the GPU while the one before them on the stream
// still runs (programmatic dependent launch).  Such a kernel sets itself up, then
// waits for everything before it, before its first access to global memory; so the order of a
// stream holds, and only the time between two kernels is saved.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gattn {

// The next kernel may be put on the GPU from here on.
__device__ __forceinline__ void let_follow() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Everything before this kernel on its stream is done, and its results can be read.
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Loads behind wait_before() of what the kernel before may have written.  Not ld.global.nc (__ldg): that is
// for data which nothing writes while the kernel runs, and this one may have been on the GPU then,
// on an SM that still holds what the same buffer had before.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load2(const void* p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
  return v;
}

// Launches a kernel that calls wait_before(); `cluster` CTAs a cluster along x (0: none).
template <class... P, class... A>
inline bool launch_following(void (*kernel)(P...), dim3 grid, dim3 block, int smem, cudaStream_t stream, int cluster, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess) return true;
  cudaGetLastError();  // reported by the return code, not to a later call
  return false;
}

}  // namespace gattn
