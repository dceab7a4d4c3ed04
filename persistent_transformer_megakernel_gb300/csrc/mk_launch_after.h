// Launch of a kernel that begins with mkw::follow_previous_kernel(): its setup overlaps the end of the stream's previous
// kernel (a decode step is a chain of short ones; measured 1 to 2 us a call).
#pragma once
#include <cuda_runtime.h>

#include "../../include/mk.h"

namespace mkw {

// cluster: CTAs of a cluster along x
template <class Params>
int launch_after(void (*kernel)(Params), dim3 grid, int threads, int smem, cudaStream_t stream, const Params &params, int cluster = 1) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, params) != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  return MK_OK;
}

}  // namespace mkw
