// launch.cuh -- programmatic dependent launch, as the training kernels use it: a kernel may
// be scheduled while the one before it on the stream finishes, and waits for that one to
// complete (dependency_wait, its first statement) before it touches memory.  The order on the
// stream is as for any launch; what is hidden is the gap between two kernels.
#pragma once

#include <cuda_runtime.h>

namespace engram {

// Waits for the kernel before this one, then lets the one after it be scheduled.
__device__ __forceinline__ void dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// cluster: CTAs a cluster (1: none).
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int64_t grid, int block, size_t smem, cudaStream_t stream,
                   int cluster, const A &...args) {
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = cluster;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attrs;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace engram
