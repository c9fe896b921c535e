// Launch with programmatic stream serialization: the kernel may start while
// the previous one on the stream finishes, so it calls pdl_wait() before its
// first global access (stream order holds for the caller as for any launch).
#pragma once
#include <utility>
#include "common.cuh"

namespace mpm {

template <typename... P, typename... A>
cudaError_t launch_serial(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                          A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace mpm
