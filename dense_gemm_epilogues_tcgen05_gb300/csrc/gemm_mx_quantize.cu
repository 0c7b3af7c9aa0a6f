// gemm_mx_quantize.cu -- rows to block-scaled numbers (OCP MX v1.0) and back.
//
//     code[i][b] = clamp(floor(log2 max_k |x[i][k]|) - emax + 127, 0, 254)   over the 32 k of block b
//     q[i][k]    = round_even(x[i][k] 2^(127 - code)), saturated
//
// with emax 2 and E2M1 elements (largest 6), or 8 and E4M3 (largest 448).  The
// multiplication by a power of two is exact, so each element is rounded once.  A
// block of zeros has code 0; one with a NaN or an infinity the NaN code 0xFF, so
// that a product shows it, and elements 0.
//
// Quantising, a thread takes 16 consecutive values, two neighbouring lanes a block
// of 32; back, 8 values.  Several pieces of a thread are on their way before the first
// is used.  Bound by HBM: 32768 x 4096 bf16 to E2M1 55 us (6.2 TB/s), and back 55 us
// (GB300, under the profiler; 110 us in turn).  With 8 values a thread the quantiser
// was bound by its instructions, 66 us; with each piece unpacked as it came, 112 us.
#include "epilogue.cuh"
#include "kernel_args.h"
#include "launch.cuh"

namespace gb300 {

namespace {

constexpr int kMxThreads = 256;
constexpr int kTo = 2, kFrom = 4;  // pieces of a thread: 16 values to codes, 8 codes to values
constexpr unsigned kAll = 0xffffffffu;

// How rows of X may be read: one value, 16 or 32 bytes at a time.
enum { kOne = 0, kSixteen = 1, kThirtyTwo = 2 };

// Sixteen values as they are stored.
template <int XT, int HOW> struct Sixteen {
    static constexpr int PV = Vec16<XT>::kPerVec, N = 16 / PV;
    uint4 u[N];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int v = 0; v < N; ++v) u[v] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const typename Elem<XT>::T *p) {
        if constexpr (HOW == kThirtyTwo) {
#pragma unroll
            for (int v = 0; v < N; v += 2)
                asm volatile("ld.global.nc.L1::no_allocate.v8.u32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(u[v].x), "=r"(u[v].y), "=r"(u[v].z), "=r"(u[v].w), "=r"(u[v + 1].x),
                               "=r"(u[v + 1].y), "=r"(u[v + 1].z), "=r"(u[v + 1].w)
                             : "l"(reinterpret_cast<const uint4 *>(p) + v));
        } else {
#pragma unroll
            for (int v = 0; v < N; ++v) u[v] = __ldg(reinterpret_cast<const uint4 *>(p) + v);
        }
    }
    __device__ __forceinline__ void unpack(float (&f)[16]) const {
#pragma unroll
        for (int v = 0; v < N; ++v) Vec16<XT>::unpack(u[v], &f[v * PV]);
    }
    // The bits of the largest |x|, as fp32: with the sign cleared values are ordered as integers, infinities and NaN
    // last; 16-bit ones two at a time.
    __device__ __forceinline__ unsigned max_bits() const {
        unsigned m = 0;
#pragma unroll
        for (int v = 0; v < N; ++v) {
            if constexpr (XT == kDtF32) {
                m = max(max(m, u[v].x & 0x7FFFFFFFu), u[v].y & 0x7FFFFFFFu);
                m = max(max(m, u[v].z & 0x7FFFFFFFu), u[v].w & 0x7FFFFFFFu);
            } else {
                m = __vimax3_u16x2(m, u[v].x & 0x7FFF7FFFu, u[v].y & 0x7FFF7FFFu);
                m = __vimax3_u16x2(m, u[v].z & 0x7FFF7FFFu, u[v].w & 0x7FFF7FFFu);
            }
        }
        if constexpr (XT == kDtF32) return m;
        m = max(m & 0xFFFFu, m >> 16);
        if constexpr (XT == kDtBF16) return m << 16;
        return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
    }
};
template <int XT> struct Sixteen<XT, kOne> {
    float v[16];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.0f;
    }
    __device__ __forceinline__ void load(const typename Elem<XT>::T *p) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = Elem<XT>::load(p + j);
    }
    __device__ __forceinline__ void unpack(float (&f)[16]) const {
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = v[j];
    }
    __device__ __forceinline__ unsigned max_bits() const {
        unsigned m = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        return m;
    }
};

// Pairs of fp32 values to E2M1 (nearest even, saturating), the first of each pair in the low nibble.
__device__ __forceinline__ uint32_t e2m1_of(const float *f) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return r;
}
__device__ __forceinline__ void e2m1_values(uint32_t c, float (&f)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}
__device__ __forceinline__ uint2 e4m3_of(const float *f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3) & 0xFFFFu;
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// Row and piece (of V values) of each of this thread's N pieces, kMxThreads apart, counted through all rows.
struct Place {
    int row, piece;  // (row M: past the end)
};
template <int V, int N>
__device__ __forceinline__ void places_of(const MxQuantArgs &a, Place (&at)[N]) {
    const unsigned per = static_cast<unsigned>(a.K) / V;
    const unsigned long long first = static_cast<unsigned long long>(blockIdx.x) * (kMxThreads * N);
    const long long row0 = first >> 32 == 0 ? static_cast<unsigned>(first) / per : first / per;
    const unsigned q = static_cast<unsigned>(first - row0 * per) + threadIdx.x, r = q / per;
    long long row = row0 + r;
    unsigned piece = q - r * per;
    const unsigned step_r = kMxThreads / per, step_p = kMxThreads - step_r * per;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        at[i] = {static_cast<int>(row < a.M ? row : a.M), static_cast<int>(piece)};
        piece += step_p;
        row += step_r;
        if (piece >= per) {
            piece -= per;
            ++row;
        }
    }
}

// QV: Q written in whole pieces' codes.
template <int ELEM, int XT, int HOW, bool QV>
__global__ void __launch_bounds__(kMxThreads) mx_quantize_kernel(const __grid_constant__ MxQuantArgs a) {
    begin_after();
    using T = typename Elem<XT>::T;
    Sixteen<XT, HOW> raw[kTo];
    Place at[kTo];
    bool live[kTo];
    int src[kTo];
    places_of<16>(a, at);
#pragma unroll
    for (int i = 0; i < kTo; ++i) {
        live[i] = at[i].row < a.M;
        src[i] = at[i].row;
        if (live[i] && a.source != nullptr) src[i] = __ldg(a.source + at[i].row);
    }
#pragma unroll
    for (int i = 0; i < kTo; ++i) {
        if (a.source != nullptr) {
            src[i] = src[i] >= 0 ? src[i] / a.top : -1;
            live[i] = live[i] && src[i] >= 0 && src[i] < a.rows_x;
        }
        raw[i].zero();
        if (live[i]) raw[i].load(static_cast<const T *>(a.X) + src[i] * a.ldx + at[i].piece * 16);
    }
#pragma unroll
    for (int i = 0; i < kTo; ++i) {
        unsigned m = raw[i].max_bits();
        m = max(m, __shfl_xor_sync(kAll, m, 1));
        constexpr int kEmax = ELEM == kMxE2M1 ? 2 : 8;
        const bool finite = m < 0x7F800000u;
        const int code = max(static_cast<int>(m >> 23) - kEmax, 0);  // (a subnormal maximum has exponent bits 0)
        const float inv = __uint_as_float(static_cast<unsigned>(254 - code) << 23);
        float f[16];
        raw[i].unpack(f);
#pragma unroll
        for (int j = 0; j < 16; j += 2) f2_unpack(f2_mul(f2_pack(f[j], f[j + 1]), f2_splat(inv)), f[j], f[j + 1]);
        if (!finite) {
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = 0.0f;
        }
        if (!live[i]) continue;
        unsigned char *q = a.Q + at[i].row * a.q_pitch + static_cast<long long>(at[i].piece) * (ELEM == kMxE2M1 ? 8 : 16);
        uint32_t w[ELEM == kMxE2M1 ? 2 : 4];
        if constexpr (ELEM == kMxE2M1) {
            w[0] = e2m1_of(f);
            w[1] = e2m1_of(f + 8);
            if constexpr (QV) *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
        } else {
            const uint2 lo = e4m3_of(f), hi = e4m3_of(f + 8);
            w[0] = lo.x; w[1] = lo.y; w[2] = hi.x; w[3] = hi.y;
            if constexpr (QV) *reinterpret_cast<uint4 *>(q) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if constexpr (!QV) {
#pragma unroll
            for (int j = 0; j < (ELEM == kMxE2M1 ? 8 : 16); ++j) q[j] = static_cast<unsigned char>(w[j / 4] >> (8 * (j & 3)));
        }
        if ((threadIdx.x & 1) == 0)
            a.scale[at[i].row * a.s_pitch + (at[i].piece >> 1)] = static_cast<unsigned char>(finite ? code : 255);
    }
}

// y[i][k] = q[i][k] 2^(code - 127), exact up to the output's rounding.
template <int ELEM, int YT, bool QV, bool YV>
__global__ void __launch_bounds__(kMxThreads) mx_dequantize_kernel(const __grid_constant__ MxQuantArgs a) {
    begin_after();
    using T = typename Elem<YT>::T;
    constexpr int PV = Vec16<YT>::kPerVec;
    uint2 w[kFrom];
    unsigned code[kFrom];
    Place at[kFrom];
    places_of<8>(a, at);
#pragma unroll
    for (int i = 0; i < kFrom; ++i) {
        w[i] = make_uint2(0, 0);
        code[i] = 0;
        if (at[i].row >= a.M) continue;
        constexpr int kBytes = ELEM == kMxE2M1 ? 4 : 8;
        const unsigned char *q = a.Q + at[i].row * a.q_pitch + static_cast<long long>(at[i].piece) * kBytes;
        if constexpr (QV) {
            if constexpr (ELEM == kMxE2M1)
                w[i].x = __ldg(reinterpret_cast<const uint32_t *>(q));
            else
                w[i] = __ldg(reinterpret_cast<const uint2 *>(q));
        } else {
#pragma unroll
            for (int j = 0; j < kBytes; ++j) (j < 4 ? w[i].x : w[i].y) |= static_cast<uint32_t>(__ldg(q + j)) << (8 * (j & 3));
        }
        code[i] = __ldg(a.scale + at[i].row * a.s_pitch + (at[i].piece >> 2));
    }
#pragma unroll
    for (int i = 0; i < kFrom; ++i) {
        if (at[i].row >= a.M) continue;
        float f[8];
        if constexpr (ELEM == kMxE2M1) {
            e2m1_values(w[i].x, f);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t two = (j < 2 ? w[i].x : w[i].y) >> (16 * (j & 1));
                const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
                const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&hr));
                f[2 * j] = t.x;
                f[2 * j + 1] = t.y;
            }
        }
        const float unit = code[i] == 255u ? NAN : __uint_as_float(code[i] == 0 ? 0x00400000u : code[i] << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= unit;
        T *y = static_cast<T *>(a.Y) + at[i].row * a.ldy + static_cast<long long>(at[i].piece) * 8;
        if constexpr (YV) {
#pragma unroll
            for (int v = 0; v < 8 / PV; ++v) reinterpret_cast<uint4 *>(y)[v] = Vec16<YT>::pack(&f[v * PV]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = Elem<YT>::cvt(f[j]);
        }
    }
}

// Blocks for M rows in pieces of `values`, `pieces` to a thread.
dim3 mx_blocks(const MxQuantArgs &a, int values, int pieces) {
    const long long n = kMxThreads * pieces;
    return dim3(static_cast<unsigned>((static_cast<long long>(a.M) * (a.K / values) + n - 1) / n));
}

template <int ELEM, int XT>
cudaError_t quantize_of(const MxQuantArgs &a, int x_bytes, bool qv, cudaStream_t s) {
    const auto kern =
        x_bytes == 32 ? (qv ? mx_quantize_kernel<ELEM, XT, kThirtyTwo, true> : mx_quantize_kernel<ELEM, XT, kThirtyTwo, false>)
        : x_bytes == 16 ? (qv ? mx_quantize_kernel<ELEM, XT, kSixteen, true> : mx_quantize_kernel<ELEM, XT, kSixteen, false>)
                        : (qv ? mx_quantize_kernel<ELEM, XT, kOne, true> : mx_quantize_kernel<ELEM, XT, kOne, false>);
    return launch_after(kern, mx_blocks(a, 16, kTo), kMxThreads, 0, s, a);
}

template <int ELEM, int YT>
cudaError_t dequantize_of(const MxQuantArgs &a, bool qv, bool yv, cudaStream_t s) {
    const auto kern = qv ? (yv ? mx_dequantize_kernel<ELEM, YT, true, true> : mx_dequantize_kernel<ELEM, YT, true, false>)
                         : (yv ? mx_dequantize_kernel<ELEM, YT, false, true> : mx_dequantize_kernel<ELEM, YT, false, false>);
    return launch_after(kern, mx_blocks(a, 8, kFrom), kMxThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_mx_quantize(int elem, int x_dtype, const MxQuantArgs &a, int x_bytes, bool q_vec, cudaStream_t s) {
    if (elem == kMxE2M1) {
        if (x_dtype == kDtF32) return quantize_of<kMxE2M1, kDtF32>(a, x_bytes, q_vec, s);
        if (x_dtype == kDtF16) return quantize_of<kMxE2M1, kDtF16>(a, x_bytes, q_vec, s);
        if (x_dtype == kDtBF16) return quantize_of<kMxE2M1, kDtBF16>(a, x_bytes, q_vec, s);
    } else if (elem == kMxE4M3) {
        if (x_dtype == kDtF32) return quantize_of<kMxE4M3, kDtF32>(a, x_bytes, q_vec, s);
        if (x_dtype == kDtF16) return quantize_of<kMxE4M3, kDtF16>(a, x_bytes, q_vec, s);
        if (x_dtype == kDtBF16) return quantize_of<kMxE4M3, kDtBF16>(a, x_bytes, q_vec, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_mx_dequantize(int elem, int y_dtype, const MxQuantArgs &a, bool q_vec, bool y_vec, cudaStream_t s) {
    if (elem == kMxE2M1) {
        if (y_dtype == kDtF32) return dequantize_of<kMxE2M1, kDtF32>(a, q_vec, y_vec, s);
        if (y_dtype == kDtF16) return dequantize_of<kMxE2M1, kDtF16>(a, q_vec, y_vec, s);
        if (y_dtype == kDtBF16) return dequantize_of<kMxE2M1, kDtBF16>(a, q_vec, y_vec, s);
    } else if (elem == kMxE4M3) {
        if (y_dtype == kDtF32) return dequantize_of<kMxE4M3, kDtF32>(a, q_vec, y_vec, s);
        if (y_dtype == kDtF16) return dequantize_of<kMxE4M3, kDtF16>(a, q_vec, y_vec, s);
        if (y_dtype == kDtBF16) return dequantize_of<kMxE4M3, kDtBF16>(a, q_vec, y_vec, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gb300
