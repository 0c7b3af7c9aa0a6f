// gemm_i8_quantize.cu -- a row of activations to 8-bit integers and one scale:
//
//     scale[i] = max_k |x[i][k]| / 127,   q[i][k] = round_even(127 x[i][k] / max_k |x[i][k]|)
//
// so q * scale is the row to within scale / 2.  A row of zeros gets scale 0
// and codes 0; a row that holds a NaN or an infinity gets a NaN scale (the
// product's row shows it) and codes 0.  127 x is exact in fp32 for 16-bit
// inputs and the quotient is correctly rounded: a 16-bit input's quotient that
// is not a tie is further from one than that rounding, so codes of 16-bit
// inputs are the exact quotient's.
//
// One block per row, one pass over memory: a thread keeps its (up to 8)
// 16-byte pieces of the row in registers between the maximum and the rounding,
// and reads what a longer row has beyond them again (from L2).
#include "grouped.cuh"

namespace gb300 {

namespace {

constexpr int kQThreads = 256, kQKeep = 8;

// |x| as an ordered integer; infinities and NaN are the largest.
__device__ __forceinline__ unsigned abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// round_even(127 x / amax).  `shrink` is 1, or 2^-32 on both where 127 x could
// overflow (exact; what it flushes is far below half a step).
__device__ __forceinline__ int code_of(float x, float amax, float shrink) {
    return __float2int_rn(__fdiv_rn(127.0f * (x * shrink), amax * shrink));
}

template <int XT, bool VEC>
__global__ void __launch_bounds__(kQThreads) i8_quantize_kernel(long long K, const void *X, long long ldx,
                                                                signed char *Q, long long ldq, float *scale) {
    using InT = typename Elem<XT>::T;
    constexpr int PV = Vec16<XT>::kPerVec;
    __shared__ unsigned part[kQThreads / 32];
    const long long row = blockIdx.x;
    const InT *x = static_cast<const InT *>(X) + row * ldx;
    signed char *q = Q + row * ldq;
    const int tid = threadIdx.x;
    unsigned m = 0u;
    uint4 keep[kQKeep];
    const long long nvec = VEC ? K / PV : 0;
    if constexpr (VEC) {
        const uint4 *xv = reinterpret_cast<const uint4 *>(x);
#pragma unroll
        for (int i = 0; i < kQKeep; ++i) {
            const long long v = tid + static_cast<long long>(i) * kQThreads;
            keep[i] = v < nvec ? __ldg(xv + v) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kQKeep; ++i) {
            float f[PV];
            Vec16<XT>::unpack(keep[i], f);
#pragma unroll
            for (int j = 0; j < PV; ++j) m = max(m, abs_bits(f[j]));
        }
        for (long long v = tid + static_cast<long long>(kQKeep) * kQThreads; v < nvec; v += kQThreads) {
            float f[PV];
            Vec16<XT>::unpack(__ldg(xv + v), f);
#pragma unroll
            for (int j = 0; j < PV; ++j) m = max(m, abs_bits(f[j]));
        }
    }
    for (long long k = nvec * PV + tid; k < K; k += kQThreads) m = max(m, abs_bits(Elem<XT>::load(x + k)));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) part[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQThreads / 32; ++w) m = max(m, part[w]);
    const bool finite = m < 0x7F800000u;
    const float amax = __uint_as_float(m);
    if (tid == 0) scale[row] = finite ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7FC00000u);
    const bool zero = !finite || m == 0u;
    const float shrink = amax >= 1.2676506e30f ? 2.3283064365386963e-10f : 1.0f;  // 2^100, 2^-32
    if constexpr (VEC) {
        const uint4 *xv = reinterpret_cast<const uint4 *>(x);
        auto store = [&](long long v, const uint4 &u) {
            float f[PV];
            Vec16<XT>::unpack(u, f);
            uint32_t w[PV / 4];
#pragma unroll
            for (int j = 0; j < PV / 4; ++j) {
                w[j] = 0u;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    w[j] |= (zero ? 0u : static_cast<uint32_t>(code_of(f[4 * j + b], amax, shrink)) & 0xFFu) << (8 * b);
            }
            if constexpr (PV == 8)
                *reinterpret_cast<uint2 *>(q + v * PV) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint32_t *>(q + v * PV) = w[0];
        };
#pragma unroll
        for (int i = 0; i < kQKeep; ++i) {
            const long long v = tid + static_cast<long long>(i) * kQThreads;
            if (v < nvec) store(v, keep[i]);
        }
        for (long long v = tid + static_cast<long long>(kQKeep) * kQThreads; v < nvec; v += kQThreads)
            store(v, __ldg(xv + v));
    }
    for (long long k = nvec * PV + tid; k < K; k += kQThreads)
        q[k] = static_cast<signed char>(zero ? 0 : code_of(Elem<XT>::load(x + k), amax, shrink));
}

template <int XT>
cudaError_t quantize_xt(long long M, long long K, const void *X, long long ldx, signed char *Q, long long ldq,
                        float *scale, cudaStream_t s) {
    const int es = static_cast<int>(sizeof(typename Elem<XT>::T));
    const bool vec = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && (M == 1 || ldx * es % 16 == 0) &&
                     (reinterpret_cast<uintptr_t>(Q) & 7u) == 0 && (M == 1 || ldq % 8 == 0);
    const unsigned grid = static_cast<unsigned>(M);
    if (vec) i8_quantize_kernel<XT, true><<<grid, kQThreads, 0, s>>>(K, X, ldx, Q, ldq, scale);
    else i8_quantize_kernel<XT, false><<<grid, kQThreads, 0, s>>>(K, X, ldx, Q, ldq, scale);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_i8_quantize(int x_dtype, long long M, long long K, const void *X, long long ldx, signed char *Q,
                               long long ldq, float *scale, cudaStream_t s) {
    if (x_dtype == kDtF32) return quantize_xt<kDtF32>(M, K, X, ldx, Q, ldq, scale, s);
    if (x_dtype == kDtF16) return quantize_xt<kDtF16>(M, K, X, ldx, Q, ldq, scale, s);
    if (x_dtype == kDtBF16) return quantize_xt<kDtBF16>(M, K, X, ldx, Q, ldq, scale, s);
    return cudaErrorInvalidValue;
}

}  // namespace gb300
