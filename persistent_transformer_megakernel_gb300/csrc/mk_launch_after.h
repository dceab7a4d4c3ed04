// Launch of a kernel that begins with mkw::follow_previous_kernel(): its setup overlaps the end of the stream's previous
// kernel (a decode step is a chain of short ones; measured 1 to 2 us a call).
#pragma once
#include <cuda_runtime.h>

#include <mutex>

#include "../../include/mk.h"

namespace mkw {

constexpr int kMaxDevices = 64;

// How a kernel can be launched on a device, looked up at its first launch there with its most dynamic shared memory:
// clusters[i] clusters of 2^(i + 1) CTAs fit on it at once.
struct Ready {
  std::once_flag once;
  bool ok = false;
  int clusters[4] = {};

  bool get(const void *fn, int threads, int smem) {
    std::call_once(once, [&] { set(fn, threads, smem); });
    return ok;
  }

 private:
  void set(const void *fn, int threads, int smem) {
    ok = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess &&
         cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    for (int i = 0; i < 4 && ok; ++i) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 2 << i;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.gridDim = dim3(2 << i);
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = smem;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&clusters[i], fn, &cfg) != cudaSuccess) clusters[i] = 0;
    }
    cudaGetLastError();
  }
};

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
