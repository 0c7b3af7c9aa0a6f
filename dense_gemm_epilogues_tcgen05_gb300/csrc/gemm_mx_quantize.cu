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
// A thread takes 8 consecutive values, four neighbouring lanes a block of 32.
// Bound by HBM; kPieces loads per thread are in flight before the first is used.
#include "epilogue.cuh"
#include "kernel_args.h"

namespace gb300 {

namespace {

constexpr int kMxThreads = 256, kPieces = 4;
constexpr unsigned kAll = 0xffffffffu;

// 16 bytes that are read once.
__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Eight values as they are stored.
template <int XT, bool VEC> struct Eight {
    static constexpr int PV = Vec16<XT>::kPerVec;
    uint4 u[8 / PV];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int v = 0; v < 8 / PV; ++v) u[v] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const typename Elem<XT>::T *p) {
#pragma unroll
        for (int v = 0; v < 8 / PV; ++v) u[v] = ld_stream(reinterpret_cast<const uint4 *>(p) + v);
    }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
#pragma unroll
        for (int v = 0; v < 8 / PV; ++v) Vec16<XT>::unpack(u[v], &f[v * PV]);
    }
    // The bits of the largest |x|, as fp32: with the sign cleared values are ordered as integers, infinities and NaN
    // last; 16-bit ones two at a time.
    __device__ __forceinline__ unsigned max_bits() const {
        unsigned m = 0;
#pragma unroll
        for (int v = 0; v < 8 / PV; ++v) {
            const uint32_t w[4] = {u[v].x, u[v].y, u[v].z, u[v].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) m = XT == kDtF32 ? max(m, w[i] & 0x7FFFFFFFu) : __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        }
        if constexpr (XT == kDtF32) return m;
        m = max(m & 0xFFFFu, m >> 16);
        if constexpr (XT == kDtBF16) return m << 16;
        return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
    }
};
template <int XT> struct Eight<XT, false> {
    float f8[8];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) f8[j] = 0.0f;
    }
    __device__ __forceinline__ void load(const typename Elem<XT>::T *p) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f8[j] = Elem<XT>::load(p + j);
    }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f8[j];
    }
    __device__ __forceinline__ unsigned max_bits() const {
        unsigned m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f8[j]) & 0x7FFFFFFFu);
        return m;
    }
};

// Pairs of fp32 values to E2M1 (nearest even, saturating), the first of each pair in the low nibble.
__device__ __forceinline__ uint32_t e2m1_of(const float (&f)[8]) {
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
__device__ __forceinline__ uint2 e4m3_of(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3) & 0xFFFFu;
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// Row and piece (of 8 values) of this thread's pieces, kMxThreads apart, counted through all rows.
struct Place {
    int row, piece;  // (row M: past the end)
};
__device__ __forceinline__ void places_of(const MxQuantArgs &a, Place (&at)[kPieces]) {
    const unsigned per = static_cast<unsigned>(a.K) / 8u;
    const long long first = static_cast<long long>(blockIdx.x) * (kMxThreads * kPieces), row0 = first / per;
    const unsigned q = static_cast<unsigned>(first - row0 * per) + threadIdx.x, r = q / per;
    long long row = row0 + r;
    unsigned piece = q - r * per;
    const unsigned step_r = kMxThreads / per, step_p = kMxThreads - step_r * per;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        at[i] = {static_cast<int>(row < a.M ? row : a.M), static_cast<int>(piece)};
        piece += step_p;
        row += step_r;
        if (piece >= per) {
            piece -= per;
            ++row;
        }
    }
}

// XV: X may be read in 16-byte pieces.  QV: Q written in whole pieces' codes.
template <int ELEM, int XT, bool XV, bool QV>
__global__ void __launch_bounds__(kMxThreads) mx_quantize_kernel(const __grid_constant__ MxQuantArgs a) {
    using T = typename Elem<XT>::T;
    Eight<XT, XV> raw[kPieces];
    Place at[kPieces];
    bool live[kPieces];
    int src[kPieces];
    places_of(a, at);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        live[i] = at[i].row < a.M;
        src[i] = at[i].row;
        if (live[i] && a.source != nullptr) src[i] = __ldg(a.source + at[i].row);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        if (a.source != nullptr) {
            src[i] = src[i] >= 0 ? src[i] / a.top : -1;
            live[i] = live[i] && src[i] >= 0 && src[i] < a.rows_x;
        }
        raw[i].zero();
        if (live[i]) raw[i].load(static_cast<const T *>(a.X) + src[i] * a.ldx + at[i].piece * 8);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        unsigned m = raw[i].max_bits();
        m = max(m, __shfl_xor_sync(kAll, m, 1));
        m = max(m, __shfl_xor_sync(kAll, m, 2));
        constexpr int kEmax = ELEM == kMxE2M1 ? 2 : 8;
        const bool finite = m < 0x7F800000u;
        const int code = max(static_cast<int>(m >> 23) - kEmax, 0);  // (a subnormal maximum has exponent bits 0)
        const float inv = __uint_as_float(static_cast<unsigned>(254 - code) << 23);
        float f[8];
        raw[i].unpack(f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) f2_unpack(f2_mul(f2_pack(f[j], f[j + 1]), f2_splat(inv)), f[j], f[j + 1]);
        if (!finite) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 0.0f;
        }
        if (!live[i]) continue;
        unsigned char *q = a.Q + at[i].row * a.q_pitch;
        if constexpr (ELEM == kMxE2M1) {
            const uint32_t w = e2m1_of(f);
            q += at[i].piece * 4;
            if constexpr (QV) {
                *reinterpret_cast<uint32_t *>(q) = w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = static_cast<unsigned char>(w >> (8 * j));
            }
        } else {
            const uint2 w = e4m3_of(f);
            q += static_cast<long long>(at[i].piece) * 8;
            if constexpr (QV) {
                *reinterpret_cast<uint2 *>(q) = w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) q[j] = static_cast<unsigned char>((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
            }
        }
        if ((threadIdx.x & 3) == 0)
            a.scale[at[i].row * a.s_pitch + (at[i].piece >> 2)] = static_cast<unsigned char>(finite ? code : 255);
    }
}

// y[i][k] = q[i][k] 2^(code - 127), exact up to the output's rounding.
template <int ELEM, int YT, bool QV, bool YV>
__global__ void __launch_bounds__(kMxThreads) mx_dequantize_kernel(const __grid_constant__ MxQuantArgs a) {
    using T = typename Elem<YT>::T;
    constexpr int PV = Vec16<YT>::kPerVec;
    uint2 w[kPieces];
    unsigned code[kPieces];
    Place at[kPieces];
    places_of(a, at);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
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
    for (int i = 0; i < kPieces; ++i) {
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

unsigned mx_blocks(const MxQuantArgs &a) {
    return static_cast<unsigned>((static_cast<long long>(a.M) * (a.K / 8) + kMxThreads * kPieces - 1) /
                                 (kMxThreads * kPieces));
}

template <int ELEM, int XT>
cudaError_t quantize_of(const MxQuantArgs &a, bool xv, bool qv, cudaStream_t s) {
    const unsigned n = mx_blocks(a);
    if (xv && qv) mx_quantize_kernel<ELEM, XT, true, true><<<n, kMxThreads, 0, s>>>(a);
    else if (xv) mx_quantize_kernel<ELEM, XT, true, false><<<n, kMxThreads, 0, s>>>(a);
    else if (qv) mx_quantize_kernel<ELEM, XT, false, true><<<n, kMxThreads, 0, s>>>(a);
    else mx_quantize_kernel<ELEM, XT, false, false><<<n, kMxThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int ELEM, int YT>
cudaError_t dequantize_of(const MxQuantArgs &a, bool qv, bool yv, cudaStream_t s) {
    const unsigned n = mx_blocks(a);
    if (qv && yv) mx_dequantize_kernel<ELEM, YT, true, true><<<n, kMxThreads, 0, s>>>(a);
    else if (qv) mx_dequantize_kernel<ELEM, YT, true, false><<<n, kMxThreads, 0, s>>>(a);
    else if (yv) mx_dequantize_kernel<ELEM, YT, false, true><<<n, kMxThreads, 0, s>>>(a);
    else mx_dequantize_kernel<ELEM, YT, false, false><<<n, kMxThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_quantize(int elem, int x_dtype, const MxQuantArgs &a, bool x_vec, bool q_vec, cudaStream_t s) {
    if (elem == kMxE2M1) {
        if (x_dtype == kDtF32) return quantize_of<kMxE2M1, kDtF32>(a, x_vec, q_vec, s);
        if (x_dtype == kDtF16) return quantize_of<kMxE2M1, kDtF16>(a, x_vec, q_vec, s);
        if (x_dtype == kDtBF16) return quantize_of<kMxE2M1, kDtBF16>(a, x_vec, q_vec, s);
    } else if (elem == kMxE4M3) {
        if (x_dtype == kDtF32) return quantize_of<kMxE4M3, kDtF32>(a, x_vec, q_vec, s);
        if (x_dtype == kDtF16) return quantize_of<kMxE4M3, kDtF16>(a, x_vec, q_vec, s);
        if (x_dtype == kDtBF16) return quantize_of<kMxE4M3, kDtBF16>(a, x_vec, q_vec, s);
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
