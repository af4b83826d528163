// Kernel launches that may begin before the stream's previous kernel has ended
// (programmatic dependent launch), and launches of clusters.
#pragma once

#include <cuda_runtime.h>

namespace fa {

// A kernel launched early runs up to its grid_wait() (sm103.cuh) while the previous kernel
// of the stream still runs, if that one has called grid_launch_dependents(), or right
// after it: its launch and prologue cost the stream little. Before grid_wait() it must
// neither read nor write what another kernel may write or read. Nor may it read through the
// read-only path, before grid_wait() or behind it: __ldg and const __restrict__ pointers
// promise that nobody writes the data while the kernel runs, which is not so while the
// previous kernel still does, and the compiler may move such loads across grid_wait().
// Ordinary loads are as fast, if no barrier arrival (a release, which waits for them) comes
// right behind. A persistent kernel with a block on every SM lets the next one start only
// when it ends: with the blocks of the next one placed as SMs came free, packed training of
// 16384 rows took 4 % longer.
template <class... P, class... A>
cudaError_t launch_as(void (*kernel)(P...), unsigned grid, int threads, int smem,
                      cudaStream_t stream, bool early, unsigned cluster, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  if (early) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, int threads, int smem,
                         cudaStream_t stream, A... args) {
  return launch_as(kernel, grid, threads, smem, stream, true, 1, args...);
}

}  // namespace fa
