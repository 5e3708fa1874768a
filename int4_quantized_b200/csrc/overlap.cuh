// overlap.cuh -- kernels whose launch and set-up overlap the kernel before them on the stream.
#pragma once

#include "common.cuh"

namespace q4 {

// The start of a kernel launched by launch_overlapped, before it touches global memory: all that
// was enqueued before it is done when this returns. Only then may the next kernel come on, so
// that one which reads its weights without waiting (Q4_QGEMM_WEIGHTS_STATIC) finds what was
// written by any kernel before this one.
Q4_DEVINL void begin_overlapped() {
    grid_dep_wait();
    grid_dep_launch();
}
// Launches a kernel (host side) that may come on while the one before it on the stream still
// runs: the kernel calls begin_overlapped() before it touches global memory, so results are
// those of launches one after the other, and only launch and set-up overlap.
template <typename... P, typename... A>
inline cudaError_t launch_overlapped(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st,
                                     unsigned cluster, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace q4
