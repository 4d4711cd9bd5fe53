// Launches of the kernels beside the products.
#pragma once
#include <cuda_runtime.h>

namespace axonn {

// Launches `kernel` on a grid, in clusters of `cluster` blocks with `shared`
// bytes of dynamic shared memory; with pdl it may start while the previous
// kernel in the stream finishes, for which it waits itself
// (griddepcontrol.wait) before it touches memory.
template <class... P, class... A>
cudaError_t launch_clusters(void (*kernel)(P...), dim3 grid, unsigned cluster, unsigned threads, bool pdl,
                            cudaStream_t stream, size_t shared, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (pdl) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// The same without clusters.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, bool pdl, cudaStream_t stream,
                         A... args) {
  return launch_clusters(kernel, grid, 1, threads, pdl, stream, 0, args...);
}

}  // namespace axonn
