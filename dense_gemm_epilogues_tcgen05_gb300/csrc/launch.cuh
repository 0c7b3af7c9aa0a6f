// launch.cuh -- launching the small kernels around the products: many of them
// follow one another, each a few microseconds long.
#pragma once

#include <cuda_runtime.h>

#include "sm103_ptx.cuh"

namespace gb300 {

// Begins every kernel launched by launch_after, which touches its shared memory at
// most before it: the grids before it in the stream are done and their memory is
// visible to the thread that waited; the next grid may be set up meanwhile.
__device__ __forceinline__ void begin_after() {
    grid_dep_wait();
    grid_dep_launch();
}

// Launches `kernel`, which begins with begin_after, so that its blocks are set up
// while the grid before it in the stream ends.
template <typename Args>
cudaError_t launch_after(void (*kernel)(const Args), dim3 grid, int threads, int smem, cudaStream_t stream,
                         const Args &args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace gb300
