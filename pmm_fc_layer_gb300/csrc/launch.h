// Launches of the kernels beside the products.
#pragma once
#include <cuda_runtime.h>

namespace axonn {

// Launches `kernel` on a grid; with pdl it may start while the previous
// kernel in the stream finishes, for which it waits itself
// (griddepcontrol.wait) before it touches memory.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, bool pdl, cudaStream_t stream,
                         A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace axonn
