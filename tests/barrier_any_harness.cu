// Test aid: barrier_any under the few-row kernel's conditions.  512 threads walk
// `rounds` rounds of a plain barrier and a vote on a flag that a thread outside the
// barrier raises after `delay` clocks; left[block * 512 + i] is the round in which
// thread i left.  Every loop ends by itself: the walk after `rounds`, the delay after
// its clocks.
#include "kernel_args.h"
#include "sm103_ptx.cuh"

namespace {

__global__ void walk(int rounds, long long delay, int *left) {
    __shared__ volatile int flag;
    if (threadIdx.x == 0) flag = 0;
    __syncthreads();
    if (threadIdx.x >= 512) {
        if (threadIdx.x == 512) {
            const long long t0 = clock64(), wait = delay * (1 + blockIdx.x % 37);
            while (clock64() - t0 < wait) {
            }
            flag = 1;
        }
        return;
    }
    int i = 0;
    for (; i < rounds; ++i) {
        asm volatile("bar.sync 1, 512;" ::: "memory");
        if (gb300::barrier_any<1, 512>(flag != 0)) break;
    }
    left[blockIdx.x * 512 + threadIdx.x] = i;
}

}  // namespace

extern "C" int run_walk(int blocks, int rounds, long long delay, int *left) {
    if (delay > 1000000) return -1;
    walk<<<blocks, 544>>>(rounds, delay, left);
    const cudaError_t e = cudaGetLastError();
    return static_cast<int>(e != cudaSuccess ? e : cudaDeviceSynchronize());
}
