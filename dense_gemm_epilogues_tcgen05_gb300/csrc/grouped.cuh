// grouped.cuh -- what the expert-grouped and 8-bit integer kernels share: the
// group table (ragged row ranges, from offsets that live on the device), the
// walk over its tiles, and the epilogue of one output.
//
// A mixture of experts sends each row (token) to some experts; sorted by
// expert, the rows of expert g are rows offsets[g] .. offsets[g+1] - 1 of one
// array.  The counts are only known on the device, so every kernel derives its
// tiles from `offsets` itself and the host never waits for them.
#pragma once

#include "epilogue.cuh"
#include "kernel_args.h"
#include "sm103_ptx.cuh"

namespace gb300 {

// The row range of every group and the number of row tiles before it, in
// shared memory: G + 1 ints of `first` (first[G] the total), G each of lo, hi.
struct GroupTable {
    int *first, *lo, *hi;
    int G;
};

__host__ __device__ constexpr int group_table_bytes(int G) { return 4 * (3 * G + 1); }

// Fill the table (every thread of the block calls this; `n` threads, a
// multiple of 32).  tiles_of(rows) is the number of row tiles of a group.
// Offsets are clamped to [0, M] and to be non-decreasing inside a group, so
// whatever the array holds, no row outside 0 .. M-1 is ever touched.
// offsets == NULL: one group of all M rows.
template <typename F>
__device__ __forceinline__ GroupTable group_table_build(int *smem, const int *offsets, int G, int M, int tid, int n,
                                                        F tiles_of) {
    GroupTable t{smem, smem + G + 1, smem + 2 * G + 1, G};
    for (int g = tid; g < G; g += n) {
        int lo = 0, hi = M;
        if (offsets != nullptr) {
            lo = min(max(__ldg(offsets + g), 0), M);
            hi = min(max(__ldg(offsets + g + 1), lo), M);
        }
        t.lo[g] = lo;
        t.hi[g] = hi;
        t.first[g + 1] = tiles_of(hi - lo);
    }
    if (tid == 0) t.first[0] = 0;
    __syncthreads();
    if (tid < 32) {
        int base = 0;
        for (int g0 = 0; g0 < G; g0 += 32) {
            const int g = g0 + tid;
            int v = g < G ? t.first[g + 1] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, v, d);
                if (tid >= d) v += o;
            }
            if (g < G) t.first[g + 1] = base + v;
            base += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
    return t;
}

// The group that row tile `t` (0 <= t < first[G]) belongs to.
__device__ __forceinline__ int group_of(const GroupTable &t, int tile) {
    int lo = 0, hi = t.G - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid + 1] > tile)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// One output: z = alpha * scale * acc (+ beta * C) (+ bias), activation, cast.
// The accurate activation forms for every output type: the cheap ones are
// within 4e-4 |z|, which shows where the activation's value is far below |z|.
template <int OUT>
__device__ __forceinline__ float grouped_value(float acc, float scale, float beta, float c_in, float bias, int epi) {
    float z = acc * scale;
    if (beta != 0.0f) z = fmaf(beta, c_in, z);
    return activate_one<OUT>(z + bias, epi, true);
}

// ------------------------------------------------------------ operand types --
template <int AB> struct SimtAcc { using T = float; };
template <> struct SimtAcc<kDtI8> { using T = int; };

template <int AB> struct SimtLoad {
    using InT = typename Elem<AB>::T;
    static __device__ __forceinline__ float load(const void *p, long long i) {
        return Elem<AB>::load(static_cast<const InT *>(p) + i);
    }
};
template <> struct SimtLoad<kDtI8> {
    static __device__ __forceinline__ int load(const void *p, long long i) {
        return static_cast<const signed char *>(p)[i];
    }
};

}  // namespace gb300
