// gemm_grouped_simt.cu -- grouped products on the CUDA cores, for the calls
// the tensor-core kernels do not take (fp32 inputs, operands whose base or
// strides TMA cannot read, K == 0): any strides, any sizes.
//
//   grouped_simt_kernel: C[r][j] = act(alpha * rs[r] * cs[g][j] * sum_k
//       A[r][k] B[g][k][j] + beta * C[r][j] + bias[g][j]), r in group g.
//       fp32 multiply-adds, k ascending; 8-bit integers in 32-bit integers.
//   wgrad_simt_kernel: C[g][m][n] = alpha * sum_r A[r][m] D[r][n] + beta * C.
//   grouped_colsum_kernel: a_sum[g][m] = alpha * sum_r A[r][m] + beta * a_sum.
//
// A block owns 64 x 64 outputs, 4 x 4 per thread, and walks 16-deep slices of
// the summed index through shared memory; operands are read along whichever
// index has stride 1.
#include "grouped.cuh"

namespace gb300 {

namespace {

constexpr int kGT = 64, kGK = 16, kGThreads = 256;

// One 16-deep slice of a 64-wide operand tile into s[k][i]: element (i, k) at
// base + i*si + k*sk, zero outside i < ni, k < nk.
template <int AB>
__device__ __forceinline__ void load_slice(typename SimtAcc<AB>::T (*s)[kGT + 1], const void *p, long long base,
                                           long long si, long long sk, int ni, int nk) {
    const bool k_fast = sk == 1;
    for (int e = threadIdx.x; e < kGT * kGK; e += kGThreads) {
        const int i = k_fast ? e / kGK : e % kGT;
        const int k = k_fast ? e % kGK : e / kGT;
        s[k][i] = (i < ni && k < nk) ? SimtLoad<AB>::load(p, base + i * si + k * sk) : 0;
    }
}

template <typename T>
__device__ __forceinline__ void slice_product(T (&acc)[4][4], const T (*a)[kGT + 1], const T (*b)[kGT + 1], int ty,
                                              int tx) {
#pragma unroll
    for (int k = 0; k < kGK; ++k) {
        T av[4], bv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = a[k][ty + 16 * i];
#pragma unroll
        for (int j = 0; j < 4; ++j) bv[j] = b[k][tx + 16 * j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4 && static_cast<T>(0.5f) != static_cast<T>(0))
                    acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
                else
                    acc[i][j] += av[i] * bv[j];
            }
    }
}

struct RowTiles64 {
    __device__ int operator()(int rows) const { return (rows + kGT - 1) / kGT; }
};

template <int AB, int OUT>
__global__ void __launch_bounds__(kGThreads) grouped_simt_kernel(const GroupedArgs a) {
    using AccT = typename SimtAcc<AB>::T;
    using OutT = typename Elem<OUT>::T;
    __shared__ AccT As[kGK][kGT + 1], Bs[kGK][kGT + 1];
    __shared__ int table[3 * kMaxGroups + 1];
    const GroupTable t = group_table_build(table, a.offsets, a.G, a.M, threadIdx.x, kGThreads, RowTiles64());
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int tiles_n = (a.N + kGT - 1) / kGT;
    const long long tiles = static_cast<long long>(t.first[a.G]) * tiles_n;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int rt = static_cast<int>(tile / tiles_n), n0 = static_cast<int>(tile % tiles_n) * kGT;
        const int g = group_of(t, rt);
        const int r0 = t.lo[g] + (rt - t.first[g]) * kGT, rows = min(kGT, t.hi[g] - r0), cols = min(kGT, a.N - n0);
        AccT acc[4][4] = {};
        for (int k0 = 0; k0 < a.K; k0 += kGK) {
            load_slice<AB>(As, a.A, r0 * a.sam + k0 * a.sak, a.sam, a.sak, rows, a.K - k0);
            load_slice<AB>(Bs, a.B, g * a.sbg + n0 * a.sbn + k0 * a.sbk, a.sbn, a.sbk, cols, a.K - k0);
            __syncthreads();
            slice_product<AccT>(acc, As, Bs, ty, tx);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
            if (r >= rows) continue;
            OutT *c = static_cast<OutT *>(a.C) + (r0 + r) * a.ldc + n0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = tx + 16 * j;
                if (n >= cols) continue;
                const long long col = static_cast<long long>(g) * a.N + n0 + n;
                const float s = product_factor(a.alpha, a.col_scale != nullptr ? a.col_scale + col : nullptr,
                                               a.row_scale != nullptr ? a.row_scale + r0 + r : nullptr);
                const float b = a.epilogue != kEpiNone ? a.bias[col] : 0.0f;
                const float cin = a.beta != 0.0f ? Elem<OUT>::load(c + n) : 0.0f;
                // no k (K == 0, alpha == 0): the scales are not read into the result
                const float p = a.K == 0 ? 0.0f : static_cast<float>(acc[i][j]);
                c[n] = Elem<OUT>::cvt(grouped_value<OUT>(p, a.K == 0 ? 0.0f : s, a.beta, cin, b, a.epilogue));
            }
        }
    }
}

template <int AB, int OUT>
__global__ void __launch_bounds__(kGThreads) wgrad_simt_kernel(const WgradArgs a) {
    using OutT = typename Elem<OUT>::T;
    __shared__ float As[kGK][kGT + 1], Ds[kGK][kGT + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int tiles_n = (a.N + kGT - 1) / kGT, tiles_m = (a.M + kGT - 1) / kGT;
    const long long per_group = static_cast<long long>(tiles_n) * tiles_m, tiles = per_group * a.G;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int g = static_cast<int>(tile / per_group);
        const long long in = tile % per_group;
        const int m0 = static_cast<int>(in / tiles_n) * kGT, n0 = static_cast<int>(in % tiles_n) * kGT;
        const int lo = min(max(a.offsets[g], 0), a.T), hi = min(max(a.offsets[g + 1], lo), a.T);
        const int ms = min(kGT, a.M - m0), ns = min(kGT, a.N - n0);
        float acc[4][4] = {};
        if (a.alpha != 0.0f) {
            for (int r0 = lo; r0 < hi; r0 += kGK) {
                load_slice<AB>(As, a.A, r0 * a.sar + m0 * a.sam, a.sam, a.sar, ms, hi - r0);
                load_slice<AB>(Ds, a.D, r0 * a.sdr + n0 * a.sdn, a.sdn, a.sdr, ns, hi - r0);
                __syncthreads();
                slice_product<float>(acc, As, Ds, ty, tx);
                __syncthreads();
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = ty + 16 * i, n = tx + 16 * j;
                if (m >= ms || n >= ns) continue;
                OutT *c = static_cast<OutT *>(a.C) + g * a.scg + (m0 + m) * a.ldc + n0 + n;
                float z = a.alpha * acc[i][j];
                if (a.beta != 0.0f) z = fmaf(a.beta, Elem<OUT>::load(c), z);
                *c = Elem<OUT>::cvt(z);
            }
    }
}

// 32 columns by 8 row lanes per block; the eight partial sums of a column meet
// in shared memory, so the order of additions is fixed.
template <int AB>
__global__ void __launch_bounds__(256) grouped_colsum_kernel(const WgradArgs a) {
    __shared__ float part[8][33];
    const int c = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int m = blockIdx.x * 32 + c, g = blockIdx.y;
    const int lo = min(max(a.offsets[g], 0), a.T), hi = min(max(a.offsets[g + 1], lo), a.T);
    float s = 0.0f;
    if (m < a.M && a.alpha != 0.0f)
        for (int r = lo + y; r < hi; r += 8) s += SimtLoad<AB>::load(a.A, r * a.sar + m * a.sam);
    part[y][c] = s;
    __syncthreads();
    if (y == 0 && m < a.M) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][c];
        float *out = a.a_sum + static_cast<long long>(g) * a.M + m;
        *out = a.beta != 0.0f ? fmaf(a.beta, *out, a.alpha * s) : a.alpha * s;
    }
}

// The same for 16-bit values contiguous along m in 16-byte aligned rows: a
// block sums 64 columns of one group, 8 per thread by LANES row lanes, four
// rows of each in flight; the lanes' sums meet in shared memory in a fixed order.
// 16384 x 2048 bf16 in 16 groups on GB300: 18 us (3.6 TB/s).
template <int AB, int LANES>
__global__ void __launch_bounds__(8 * LANES) grouped_colsum_vec_kernel(const WgradArgs a) {
    __shared__ float part[LANES][64 + 8];
    const int cv = threadIdx.x & 7, y = threadIdx.x >> 3;
    const int g = blockIdx.y, m0 = blockIdx.x * 64, m = m0 + cv * 8;
    grid_dep_launch();  // the product's kernel may set itself up meanwhile; it waits for this grid
    const int lo = min(max(a.offsets[g], 0), a.T), hi = min(max(a.offsets[g + 1], lo), a.T);
    float s[8] = {};
    if (m + 8 <= a.M) {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const typename Elem<AB>::T *>(a.A) + m);
        const long long pitch = a.sar / 8;
        int r = lo + y;
        for (; hi - r > 3 * LANES; r += 4 * LANES) {
            uint4 u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = __ldg(src + (r + i * LANES) * pitch);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float f[8];
                Vec16<AB>::unpack(u[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] += f[j];
            }
        }
        for (; r < hi; r += LANES) {
            float f[8];
            Vec16<AB>::unpack(__ldg(src + r * pitch), f);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] += f[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            for (int r = lo + y; m + j < a.M && r < hi; r += LANES) s[j] += SimtLoad<AB>::load(a.A, r * a.sar + m + j);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) part[y][cv * 8 + j] = s[j];
    __syncthreads();
    const int c = threadIdx.x, col = m0 + c;
    if (c < 64 && col < a.M) {
        float sum = part[0][c];
#pragma unroll
        for (int i = 1; i < LANES; ++i) sum += part[i][c];
        float *out = a.a_sum + static_cast<long long>(g) * a.M + col;
        *out = a.beta != 0.0f ? fmaf(a.beta, *out, a.alpha * sum) : a.alpha * sum;
    }
}

template <int AB>
cudaError_t launch_colsum_vec(const WgradArgs &a, int sms, cudaStream_t s) {
    const dim3 grid((a.M + 63) / 64, a.G);
    // A block's time is its group's rows over its lanes, four loads at a time: many lanes for long groups, and
    // where there are few blocks (16 groups of some 1000 rows x 2048 columns on GB300: 34 us with 32 lanes).
    if (static_cast<long long>(grid.x) * grid.y < 2ll * sms || a.T / a.G >= 256)
        grouped_colsum_vec_kernel<AB, 128><<<grid, 1024, 0, s>>>(a);
    else
        grouped_colsum_vec_kernel<AB, 32><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

template <int AB>
cudaError_t grouped_simt_out(int out, const GroupedArgs &a, int grid, cudaStream_t s) {
    if (out == kDtF32) grouped_simt_kernel<AB, kDtF32><<<grid, kGThreads, 0, s>>>(a);
    else if (out == kDtF16) grouped_simt_kernel<AB, kDtF16><<<grid, kGThreads, 0, s>>>(a);
    else if (out == kDtBF16) grouped_simt_kernel<AB, kDtBF16><<<grid, kGThreads, 0, s>>>(a);
    else return cudaErrorInvalidValue;
    return cudaGetLastError();
}

template <int AB>
cudaError_t wgrad_simt_out(int out, const WgradArgs &a, int grid, cudaStream_t s) {
    if (out == kDtF32) wgrad_simt_kernel<AB, kDtF32><<<grid, kGThreads, 0, s>>>(a);
    else if (out == kDtF16) wgrad_simt_kernel<AB, kDtF16><<<grid, kGThreads, 0, s>>>(a);
    else if (out == kDtBF16) wgrad_simt_kernel<AB, kDtBF16><<<grid, kGThreads, 0, s>>>(a);
    else return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_simt(int ab, int out, const GroupedArgs &a, int grid, cudaStream_t s) {
    if (ab == kDtF32) return out == kDtF32 ? grouped_simt_out<kDtF32>(out, a, grid, s) : cudaErrorInvalidValue;
    if (ab == kDtF16) return grouped_simt_out<kDtF16>(out, a, grid, s);
    if (ab == kDtBF16) return grouped_simt_out<kDtBF16>(out, a, grid, s);
    if (ab == kDtI8) return grouped_simt_out<kDtI8>(out, a, grid, s);
    return cudaErrorInvalidValue;
}

cudaError_t launch_wgrad_simt(int ab, int out, const WgradArgs &a, int grid, cudaStream_t s) {
    if (ab == kDtF32) return out == kDtF32 ? wgrad_simt_out<kDtF32>(out, a, grid, s) : cudaErrorInvalidValue;
    if (ab == kDtF16) return wgrad_simt_out<kDtF16>(out, a, grid, s);
    if (ab == kDtBF16) return wgrad_simt_out<kDtBF16>(out, a, grid, s);
    return cudaErrorInvalidValue;
}

cudaError_t launch_grouped_colsum(int ab, const WgradArgs &a, bool vec, int sms, cudaStream_t s) {
    if (vec && ab == kDtF16) return launch_colsum_vec<kDtF16>(a, sms, s);
    if (vec && ab == kDtBF16) return launch_colsum_vec<kDtBF16>(a, sms, s);
    const dim3 grid((a.M + 31) / 32, a.G);
    if (ab == kDtF32) grouped_colsum_kernel<kDtF32><<<grid, 256, 0, s>>>(a);
    else if (ab == kDtF16) grouped_colsum_kernel<kDtF16><<<grid, 256, 0, s>>>(a);
    else if (ab == kDtBF16) grouped_colsum_kernel<kDtBF16><<<grid, 256, 0, s>>>(a);
    else return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace gb300
