// Kernel launches shared by the translation units.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace twell {

// Launch with programmatic stream serialisation: the kernel may be scheduled
// while the previous kernel in the stream is still running.  Every kernel of
// this library issues griddepcontrol.wait before its first global memory
// access, so ordering is kept; only the launch and set-up overlap.
template <class... KArgs, class... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, int block, size_t smem, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// launch_pdl for clusters of `cluster` CTAs.
template <class... KArgs, class... Args>
cudaError_t launch_pdl_cluster(int cluster, void (*kern)(KArgs...), int grid, int block, size_t smem, cudaStream_t s,
                               Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// launch_pdl for clusters of two CTAs.
template <class... KArgs, class... Args>
cudaError_t launch_pdl_pair(void (*kern)(KArgs...), int grid, int block, size_t smem, cudaStream_t s,
                            Args&&... args) {
  return launch_pdl_cluster(2, kern, grid, block, smem, s, std::forward<Args>(args)...);
}

}  // namespace twell
