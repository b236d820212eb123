// launch.cuh -- host-side launch helper shared by the cache and position kernels.
#pragma once

#include "common.cuh"

namespace fa {

// Accessors defined in api.cu.
unsigned* device_error_word();
int device_sm_count();
unsigned long long wait_timeout_ns();

// Launches `kfn` as a programmatic dependent of the launch before it on `stream`, in
// clusters of `cluster` blocks: the kernel executes griddepcontrol.wait before its first
// global access.
template <typename... KArgs, typename... Args>
inline int launch_dependent_cluster(void (*kfn)(KArgs...), dim3 grid, int cluster, dim3 block, size_t smem,
                                    cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kfn, args...);
  if (e != cudaSuccess) return record_cuda_failure(e);
  return launch_status();
}
template <typename... KArgs, typename... Args>
inline int launch_dependent(void (*kfn)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                            const Args&... args) {
  return launch_dependent_cluster(kfn, grid, 1, block, smem, stream, args...);
}

// Whether two byte ranges share a byte (a null pointer: no).
inline bool overlap(const void* a, long long a_bytes, const void* b, long long b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x && y && x < y + static_cast<uintptr_t>(b_bytes) && y < x + static_cast<uintptr_t>(a_bytes);
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Only after pdl_wait(): a dependent launched early must not see the grid before this
// one as complete while it still runs.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace fa
