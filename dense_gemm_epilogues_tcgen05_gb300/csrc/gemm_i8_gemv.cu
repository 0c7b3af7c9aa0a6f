// gemm_i8_gemv.cu -- 8-bit integer products for few rows (decoding): the
// weights are read once, straight into registers, and everything else hides
// behind that.
//
// A block takes 16 rows of W (output channels) and up to 8 rows of X; its eight
// warps split K.  The products are mma.sync m16n8k32 on the codes, summed in
// 32-bit integers: exact, and in any order the same.  The sum over k does not
// care which k an MMA's slot holds as long as both operands agree, so a lane
// loads 16 consecutive codes of its two rows of W (row g = lane / 4 and g + 8)
// and of its row of X (row g), at k = 64 step + 16 (lane % 4), and feeds words
// 0, 1 to one MMA and 2, 3 to the next: whole 16-byte loads, no shuffles.
//
// Bound: HBM, by the weights' bytes.
#include "grouped.cuh"

namespace gb300 {

namespace {

constexpr int kGvWarps = 8, kGvRowsW = 16, kGvRowsX = 8, kGvUnroll = 4;

__device__ __forceinline__ uint4 ldg_stream(const void *p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// Codes k .. k+15 of a row of K; zero from K on (bytes past K are not read).
template <bool STREAM>
__device__ __forceinline__ uint4 codes16(const signed char *row, int k, int K) {
    if (k + 16 <= K) return STREAM ? ldg_stream(row + k) : __ldg(reinterpret_cast<const uint4 *>(row + k));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (k + i < K) w[i >> 2] |= static_cast<uint32_t>(static_cast<unsigned char>(row[k + i])) << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int OUT>
__global__ void __launch_bounds__(kGvWarps * 32) i8_gemv_kernel(const GroupedArgs a) {
    using OutT = typename Elem<OUT>::T;
    extern __shared__ int table[];
    __shared__ int part[kGvWarps][kGvRowsW * kGvRowsX];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g8 = lane >> 2, t4 = lane & 3;
    GroupTable t{};
    int row_tiles = (a.M + kGvRowsX - 1) / kGvRowsX;
    if (a.offsets != nullptr) {
        t = group_table_build(table, a.offsets, a.G, a.M, threadIdx.x, kGvWarps * 32, RowTilesOf{kGvRowsX});
        row_tiles = t.first[a.G];
    }
    const int tiles_n = (a.N + kGvRowsW - 1) / kGvRowsW;
    const long long tiles = static_cast<long long>(row_tiles) * tiles_n;
    const int steps = (a.K + 63) / 64;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int rt = static_cast<int>(tile / tiles_n), n0 = static_cast<int>(tile - static_cast<long long>(rt) * tiles_n) * kGvRowsW;
        int g = 0, r0 = rt * kGvRowsX, hi = a.M;
        if (a.offsets != nullptr) {
            g = group_of(t, rt);
            r0 = t.lo[g] + (rt - t.first[g]) * kGvRowsX;
            hi = t.hi[g];
        }
        const int nr = min(kGvRowsX, hi - r0);
        // rows past the edge re-read one inside (never stored); rows of X past the group count as zero
        const signed char *W = static_cast<const signed char *>(a.B) + g * a.sbg;
        const signed char *w0 = W + static_cast<long long>(min(n0 + g8, a.N - 1)) * a.sbn;
        const signed char *w1 = W + static_cast<long long>(min(n0 + g8 + 8, a.N - 1)) * a.sbn;
        const signed char *x = static_cast<const signed char *>(a.A) + static_cast<long long>(r0 + min(g8, nr - 1)) * a.sam;
        const bool x_ok = g8 < nr;
        int d[4] = {0, 0, 0, 0};
        for (int s = warp; s < steps; s += kGvWarps * kGvUnroll) {
            uint4 p[kGvUnroll], q[kGvUnroll], v[kGvUnroll];
#pragma unroll
            for (int u = 0; u < kGvUnroll; ++u) {
                const int k = (s + u * kGvWarps) * 64 + t4 * 16;
                p[u] = codes16<true>(w0, k, a.K);
                q[u] = codes16<true>(w1, k, a.K);
            }
#pragma unroll
            for (int u = 0; u < kGvUnroll; ++u) {
                const int k = (s + u * kGvWarps) * 64 + t4 * 16;
                v[u] = x_ok ? codes16<false>(x, k, a.K) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < kGvUnroll; ++u) {
                mma_s8(d, p[u].x, q[u].x, p[u].y, q[u].y, v[u].x, v[u].y);
                mma_s8(d, p[u].z, q[u].z, p[u].w, q[u].w, v[u].z, v[u].w);
            }
        }
        // d: rows of W g8, g8 + 8; rows of X 2 t4, 2 t4 + 1
        part[warp][(2 * t4) * kGvRowsW + g8] = d[0];
        part[warp][(2 * t4 + 1) * kGvRowsW + g8] = d[1];
        part[warp][(2 * t4) * kGvRowsW + g8 + 8] = d[2];
        part[warp][(2 * t4 + 1) * kGvRowsW + g8 + 8] = d[3];
        __syncthreads();
        const int i = threadIdx.x;
        if (i < kGvRowsW * kGvRowsX) {
            const int r = i / kGvRowsW, n = n0 + i % kGvRowsW;
            int sum = 0;
#pragma unroll
            for (int w = 0; w < kGvWarps; ++w) sum += part[w][i];
            if (r < nr && n < a.N) {
                const long long gn = static_cast<long long>(g) * a.N + n;
                float s = a.alpha;
                if (a.col_scale != nullptr) s *= a.col_scale[gn];
                if (a.row_scale != nullptr) s *= a.row_scale[r0 + r];
                OutT *c = static_cast<OutT *>(a.C) + (r0 + r) * a.ldc + n;
                const float bias = a.epilogue != kEpiNone ? a.bias[gn] : 0.0f;
                const float cin = a.beta != 0.0f ? Elem<OUT>::load(c) : 0.0f;
                *c = Elem<OUT>::cvt(grouped_value<OUT>(static_cast<float>(sum), s, a.beta, cin, bias, a.epilogue));
            }
        }
        __syncthreads();
    }
}

template <int OUT>
cudaError_t launch_gemv_out(const GroupedArgs &a, int sms, cudaStream_t s) {
    const long long row_tiles = (a.M + kGvRowsX - 1) / kGvRowsX + (a.offsets != nullptr ? a.G : 0);
    const long long tiles = row_tiles * ((a.N + kGvRowsW - 1) / kGvRowsW);
    const long long cap = static_cast<long long>(sms) * 4;  // blocks resident at once
    const int grid = static_cast<int>(tiles < cap ? tiles : cap);
    const size_t smem = a.offsets != nullptr ? group_table_bytes(a.G) : 0;
    i8_gemv_kernel<OUT><<<grid, kGvWarps * 32, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_i8_gemv(int out, const GroupedArgs &a, int sms, cudaStream_t s) {
    if (out == kDtF32) return launch_gemv_out<kDtF32>(a, sms, s);
    if (out == kDtF16) return launch_gemv_out<kDtF16>(a, sms, s);
    if (out == kDtBF16) return launch_gemv_out<kDtBF16>(a, sms, s);
    return cudaErrorInvalidValue;
}

}  // namespace gb300
