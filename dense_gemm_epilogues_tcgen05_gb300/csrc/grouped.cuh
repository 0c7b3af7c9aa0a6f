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
// Offsets are clamped to [0, M], and where one is below an earlier one it is
// raised to that, so whatever the array holds, no row outside 0 .. M-1 is ever
// touched, no row belongs to two groups, and the tiles of all groups together
// are no more than M rows and G groups can have (first[G] stays in 32 bits).
// offsets == NULL: one group of all M rows.
template <typename F>
__device__ __forceinline__ GroupTable group_table_build(int *smem, const int *offsets, int G, int M, int tid, int n,
                                                        F tiles_of) {
    GroupTable t{smem, smem + G + 1, smem + 2 * G + 1, G};
    bool falls = false;
    for (int g = tid; g < G; g += n) {
        int lo = 0, hi = M;
        if (offsets != nullptr) {
            lo = min(max(__ldg(offsets + g), 0), M);
            hi = min(max(__ldg(offsets + g + 1), 0), M);
            falls = falls || hi < lo;
        }
        t.lo[g] = lo;
        t.hi[g] = hi;
        t.first[g + 1] = tiles_of(max(hi - lo, 0));
    }
    if (tid == 0) t.first[0] = 0;
    if (__syncthreads_or(falls)) {  // offsets that are not non-decreasing
        if (tid == 0) {
            int end = 0;
            for (int g = 0; g < G; ++g) {
                t.lo[g] = end = max(end, t.lo[g]);
                t.hi[g] = end = max(end, t.hi[g]);
                t.first[g + 1] = tiles_of(t.hi[g] - t.lo[g]);
            }
        }
        __syncthreads();
    }
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

// ------------------------------------------------------------- row tiles --
// The tensor-core kernels give a group of n rows ceil(n / most) tiles of one
// common width, a multiple of 32 (`most` is one too).
struct RowTilesOf {
    int most;
    __device__ __forceinline__ int operator()(int rows) const { return (rows + most - 1) / most; }
};

__device__ __forceinline__ int tile_width(int n, int tiles) {
    const int per = (n + tiles - 1) / tiles;
    return (per + 31) & ~31;
}

struct GroupedTile {
    int g;          // group
    int f0;         // first column of C (256 of them)
    int r0, nr;     // first row of C (gradient: of its index m) and how many this tile stores
    int bn;         // MMA columns, nr rounded up to 32
    int k0, nk;     // gradient: first row summed and how many; forward: 0 and K
};

// Tile `tile` of a forward product: a row tile's column tiles follow one another.
__device__ __forceinline__ GroupedTile row_tile(const GroupTable &t, long long tile, int tiles_f, int K) {
    GroupedTile o;
    const int rt = static_cast<int>(tile / tiles_f);
    o.f0 = static_cast<int>(tile - static_cast<long long>(rt) * tiles_f) * 256;
    o.g = group_of(t, rt);
    const int lo = t.lo[o.g], n = t.hi[o.g] - lo, nt = t.first[o.g + 1] - t.first[o.g];
    const int w = tile_width(n, nt);
    o.r0 = lo + (rt - t.first[o.g]) * w;
    o.nr = min(w, lo + n - o.r0);
    o.bn = (o.nr + 31) & ~31;
    o.k0 = 0;
    o.nk = K;
    return o;
}

// The factor of a product's sum, (alpha * column's) * row's: one order in every
// kernel, so that an output does not depend on which of them computed it.
__device__ __forceinline__ float product_factor(float alpha, const float *col_scale, const float *row_scale) {
    float s = alpha;
    if (col_scale != nullptr) s = __fmul_rn(s, *col_scale);
    if (row_scale != nullptr) s = __fmul_rn(s, *row_scale);
    return s;
}

// One output: z = scale * acc (+ beta * C) (+ bias), activation; a rounding each,
// as chunk_values_t has them (no product contracted into the addition).
// The accurate activation forms for every output type: the cheap ones are
// within 4e-4 |z|, which shows where the activation's value is far below |z|.
template <int OUT>
__device__ __forceinline__ float grouped_value(float acc, float scale, float beta, float c_in, float bias, int epi) {
    float z = __fmul_rn(acc, scale);
    if (beta != 0.0f) z = fmaf(beta, c_in, z);
    if (epi != kEpiNone) z = __fadd_rn(z, bias);
    if (epi == kEpiBiasGelu) {
        // the form of chunk_values_t: the compiler contracts gelu_erf's 1 - q with the product q
        float unused = 0.0f;
        gelu_erf2(z, unused);
        return z;
    }
    return activate_one<OUT>(z, epi, true);
}

// ------------------------------------------------- transposed accumulators --
// The tensor-core kernels compute C^T: the weights' output channels (or, for
// the weight gradient, its contiguous index) are the MMA's rows and lie in
// tensor-memory lanes, the tokens are its columns -- so that a ragged group
// costs columns in steps of 32, not rows in steps of 256.  A warp then holds
// 32 consecutive columns of C in its lanes and 32 rows of C in its registers,
// and each store instruction writes 32 columns of a row, 64 or 128 bytes: no
// staging, any pitch and alignment, and a group's last rows need no other path.
// (27270 x 6304 fp16 outputs of a product 320 deep on GB300: 106 us; through
// shared memory as TMA boxes of 32 rows x 64 bytes 113 us, at 6 to 7 clocks per
// box row; pairing lanes for 32-bit stores 195 us; four warps joining their
// columns in shared memory for 16-byte stores 153 us.)
struct StoreArgs {
    long long ldc;
    float alpha, beta;
    int epi;
};

// v: this lane's column at 32 consecutive rows, of which the first nrow are
// valid: sums on entry, outputs before the cast on return.  c: element (row 0,
// this lane's column); the lane's column is `left` columns before the end of C's
// rows (<= 0: outside).  row_scale: of row 0 on, or NULL; col_scale and bias:
// this lane's column's.  Warp-collective.
template <int OUT>
__device__ __forceinline__ void chunk_values_t(float (&v)[32], const typename Elem<OUT>::T *c, int left, int nrow,
                                               const float *row_scale, float col_scale, float bias,
                                               const StoreArgs &e) {
    const int lane = threadIdx.x & 31;
    const bool f_ok = left > 0;
    const float a = e.alpha * col_scale;
    if (row_scale != nullptr) {
        const float rs = lane < nrow ? row_scale[lane] : 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= a * __shfl_sync(0xffffffffu, rs, j);
    } else {
        scale_alpha(v, a);
    }
    if (e.beta != 0.0f) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (f_ok && j < nrow) v[j] = fmaf(e.beta, Elem<OUT>::load(c + j * e.ldc), v[j]);
    }
    if (e.epi != kEpiNone) {
        const uint64_t b2 = f2_splat(bias);
#pragma unroll
        for (int j = 0; j < 32; j += 2) f2_unpack(f2_add(f2_pack(v[j], v[j + 1]), b2), v[j], v[j + 1]);
        if (e.epi >= kEpiBiasGelu) activate_run<OUT, 32>(v, 0, e.epi, true);
    }
}

// The outputs v from registers: 32 columns of a row per instruction.
template <int OUT>
__device__ __forceinline__ void store_chunk_t(const float (&v)[32], typename Elem<OUT>::T *c, int left, int nrow,
                                              long long ldc) {
    if (left <= 0) return;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        if (j < nrow) *c = Elem<OUT>::cvt(v[j]);
        c += ldc;
    }
}

// ------------------------------------------------------------ 8-bit codes --
// Four codes to two pairs of binary16.
__device__ __forceinline__ void expand4(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = codes ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
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
