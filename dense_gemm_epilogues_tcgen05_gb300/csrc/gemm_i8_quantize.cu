// gemm_i8_quantize.cu -- a row of activations to 8-bit integers and one scale:
//
//     scale[i] = max_k |x[i][k]| / 127,   q[i][k] = round_even(127 x[i][k] / max_k |x[i][k]|)
//
// so q * scale is the row to within scale / 2.  A row of zeros gets scale 0
// and codes 0; a row that holds a NaN or an infinity gets a NaN scale (the
// product's row shows it) and codes 0.
//
// One pass over memory: a thread keeps its (up to 8) 16-byte pieces of a row in
// registers between the maximum and the rounding.  Many rows: persistent blocks,
// which load the next row's pieces before they round a row's.  Few, very long or
// unaligned rows: one block per row, which reads what a row has beyond the pieces
// again (from L2).  The maximum of
// 16-bit values is taken on their bits, two per instruction: with the sign
// cleared, they are ordered as integers, infinities and NaN last.
//
// The codes are those of the exact quotient.  n = round(x * (127 / max)) is the
// quotient's rounding or, within 2^-15 of a tie (the product is off by at most
// 2^-23 of at most 127), a neighbour of it.  There the remainder 127 x - n max
// decides: twice its size against max, and the even code where they are equal.
// Next to a tie the fused multiply-add gives the remainder exactly (both terms
// are multiples of max's last place, or n is 0), and so does the subtraction of
// max; 127 x is exact for 16-bit inputs, and what its rounding cut off an fp32
// input's is added last.  (Ties are not rare: with x and max of few bits the
// quotients lie on a coarse grid, and in rows of normal bf16 values most warps meet one.)
//
// Bound: HBM (3 bytes per 16-bit value): 16384 x 8192 bf16 68 us on GB300, 5.9 TB/s,
// with 67 % of the issue slots used (with a division kept for extreme rows, and the
// stack it needs, 80 us; a block per row without the prefetch 103 us; a division per
// value 194 us).
#include "grouped.cuh"

namespace gb300 {

namespace {

constexpr int kQThreads = 256;

// |x| as an ordered integer; infinities and NaN are the largest.
__device__ __forceinline__ unsigned abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

struct QRow {
    float amax, inv;  // the row's maximum times pre, and 127 over that
    float pre;        // 1, or the power of two that brings a very small or large maximum near 1: its values
                      // are multiplied by it (exact where a code other than 0 can come of it)
    bool zero;        // codes 0 throughout
};

// What to add to the code n (odd or even) of x, at most one off, for
// round_even(127 x / amax); x and amax with `pre`.
template <int XT>
__device__ __forceinline__ int step_to_nearest(float x, float n, bool odd, float amax) {
    const float p = 127.0f * x, e = fmaf(-n, amax, p);
    float d = 2.0f * fabsf(e) - amax;
    if constexpr (XT == kDtF32) {
        const float cut = fmaf(127.0f, x, -p);
        d = fmaf(e > 0.0f ? 2.0f : -2.0f, cut, d);
    }
    return d > 0.0f || (d == 0.0f && odd) ? (e > 0.0f ? 1 : -1) : 0;
}

// The code of one value.
template <int XT>
__device__ __forceinline__ int code_of(float x, const QRow &row) {
    x *= row.pre;
    const int n = __float2int_rn(x * row.inv);
    return row.zero ? 0 : n + step_to_nearest<XT>(x, static_cast<float>(n), (n & 1) != 0, row.amax);
}

// The largest |x| of a 16-byte piece, as the bits of an fp32 value; 16-bit types
// two at a time (the halves of `acc` are combined at the end).
template <int XT>
__device__ __forceinline__ void max16(const uint4 &u, unsigned &acc) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (XT == kDtF32)
            acc = max(acc, w[i] & 0x7FFFFFFFu);
        else
            acc = __vmaxu2(acc, w[i] & 0x7FFF7FFFu);
    }
}

template <int XT>
__device__ __forceinline__ unsigned max_bits(unsigned acc) {
    if constexpr (XT == kDtF32) return acc;
    const unsigned m = max(acc & 0xFFFFu, acc >> 16);
    if constexpr (XT == kDtBF16) return m << 16;
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
}

// Codes of N values (N even, at most 8) into N bytes.  r + 1.5 * 2^23 holds
// round_even(r) in its low bits, as a two's complement byte.
template <int XT, int N>
__device__ __forceinline__ void codes_of(float (&f)[N], const QRow &row, uint32_t (&w)[N / 4]) {
    constexpr float kMagic = 12582912.0f;
    if (row.pre != 1.0f) {
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] *= row.pre;
    }
    uint32_t t[N];
    float worst = 0.0f;
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const uint64_t r = f2_mul(f2_pack(f[j], f[j + 1]), f2_splat(row.inv));
        const uint64_t s = f2_add(r, f2_splat(kMagic));
        const uint64_t back = f2_add(s, f2_splat(-kMagic));
        const uint64_t off = f2_fma(back, f2_splat(-1.0f), r);
        float s0, s1, o0, o1;
        f2_unpack(s, s0, s1);
        f2_unpack(off, o0, o1);
        t[j] = __float_as_uint(s0);
        t[j + 1] = __float_as_uint(s1);
        worst = fmaxf(worst, fmaxf(fabsf(o0), fabsf(o1)));
    }
    if (worst > 0.5f - 0x1p-15f) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float n = __uint_as_float(t[j]) - kMagic;
            t[j] += static_cast<uint32_t>(step_to_nearest<XT>(f[j], n, (t[j] & 1u) != 0, row.amax));
        }
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const uint32_t lo = __byte_perm(t[4 * i], t[4 * i + 1], 0x0040), hi = __byte_perm(t[4 * i + 2], t[4 * i + 3], 0x0040);
        w[i] = row.zero ? 0u : __byte_perm(lo, hi, 0x5410);
    }
}

// What a row's largest |x| (as bits) makes of it; one thread writes the scale.
__device__ __forceinline__ QRow row_scale(unsigned m, float *scale, bool writes) {
    const bool finite = m < 0x7F800000u;
    QRow r;
    const float amax = __uint_as_float(m);
    r.zero = !finite || m == 0u;
    r.pre = r.zero || (amax > 1e-30f && amax < 1e30f) ? 1.0f : amax < 1.0f ? 0x1p64f : 0x1p-64f;
    r.amax = amax * r.pre;
    r.inv = r.zero ? 0.0f : __fdiv_rn(127.0f, r.amax);
    if (writes) *scale = finite ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7FC00000u);
    return r;
}

// Codes of the 16-byte piece u, piece v of its row.
template <int XT>
__device__ __forceinline__ void store_codes(signed char *q, long long v, const uint4 &u, const QRow &r) {
    constexpr int PV = Vec16<XT>::kPerVec;
    float f[PV];
    Vec16<XT>::unpack(u, f);
    uint32_t w[PV / 4];
    codes_of<XT, PV>(f, r, w);
    if constexpr (PV == 8)
        *reinterpret_cast<uint2 *>(q + v * PV) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t *>(q + v * PV) = w[0];
}

// VEC: 16-byte loads of X and whole-word stores of Q; KEEP pieces per thread stay in registers.
template <int XT, bool VEC, int KEEP>
__global__ void __launch_bounds__(kQThreads) i8_quantize_kernel(long long K, const void *X, long long ldx,
                                                                signed char *Q, long long ldq, float *scale) {
    using InT = typename Elem<XT>::T;
    constexpr int PV = Vec16<XT>::kPerVec;
    __shared__ unsigned part[kQThreads / 32];
    const long long row = blockIdx.x;
    const InT *x = static_cast<const InT *>(X) + row * ldx;
    signed char *q = Q + row * ldq;
    const int tid = threadIdx.x, n = blockDim.x;
    const uint4 *xv = reinterpret_cast<const uint4 *>(x);
    const long long nvec = VEC ? K / PV : 0;
    unsigned acc = 0u;
    uint4 keep[KEEP];
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const long long v = tid + static_cast<long long>(i) * n;
            keep[i] = v < nvec ? __ldg(xv + v) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < KEEP; ++i) max16<XT>(keep[i], acc);
        for (long long v = tid + static_cast<long long>(KEEP) * n; v < nvec; v += n) max16<XT>(__ldg(xv + v), acc);
    }
    unsigned m = max_bits<XT>(acc);
    for (long long k = nvec * PV + tid; k < K; k += n) m = max(m, abs_bits(Elem<XT>::load(x + k)));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) part[tid >> 5] = m;
    __syncthreads();
    for (int w = 0; w < n >> 5; ++w) m = max(m, part[w]);
    const QRow r = row_scale(m, scale + row, tid == 0);
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const long long v = tid + static_cast<long long>(i) * n;
            if (v < nvec) store_codes<XT>(q, v, keep[i], r);
        }
        for (long long v = tid + static_cast<long long>(KEEP) * n; v < nvec; v += n)
            store_codes<XT>(q, v, __ldg(xv + v), r);
    }
    for (long long k = nvec * PV + tid; k < K; k += n)
        q[k] = static_cast<signed char>(code_of<XT>(Elem<XT>::load(x + k), r));
}

// Persistent form for many rows of `pieces` 16-byte pieces, at most KEEP
// blockDim.x: the next row's pieces are on their way while a row is rounded.
template <int XT, int KEEP>
__global__ void __launch_bounds__(kQThreads, KEEP <= 4 ? 4 : 3)
    i8_quantize_rows_kernel(long long M, int pieces, const void *X, long long ldx, signed char *Q, long long ldq,
                            float *scale) {
    __shared__ unsigned part[2][kQThreads / 32];
    const int tid = threadIdx.x, n = blockDim.x;
    const uint4 *x = static_cast<const uint4 *>(X);
    const long long pitch = ldx * static_cast<long long>(sizeof(typename Elem<XT>::T)) / 16;
    uint4 cur[KEEP], nxt[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        nxt[i] = tid + i * n < pieces ? __ldg(x + blockIdx.x * pitch + tid + i * n) : make_uint4(0, 0, 0, 0);
    int flip = 0;
    for (long long row = blockIdx.x; row < M; row += gridDim.x, flip ^= 1) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) cur[i] = nxt[i];
        const long long ahead = row + gridDim.x;
        if (ahead < M) {
#pragma unroll
            for (int i = 0; i < KEEP; ++i)
                if (tid + i * n < pieces) nxt[i] = __ldg(x + ahead * pitch + tid + i * n);
        }
        unsigned acc = 0u;
#pragma unroll
        for (int i = 0; i < KEEP; ++i) max16<XT>(cur[i], acc);
        unsigned m = __reduce_max_sync(0xffffffffu, max_bits<XT>(acc));
        if ((tid & 31) == 0) part[flip][tid >> 5] = m;
        __syncthreads();  // the other half of `part` is free: all have read it before this row's barrier
        for (int w = 0; w < n >> 5; ++w) m = max(m, part[flip][w]);
        const QRow r = row_scale(m, scale + row, tid == 0);
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if (tid + i * n < pieces) store_codes<XT>(Q + row * ldq, tid + i * n, cur[i], r);
    }
}

template <int XT, int KEEP>
cudaError_t quantize_keep(long long M, int threads, long long K, const void *X, long long ldx, signed char *Q,
                          long long ldq, float *scale, int sms, cudaStream_t s) {
    const long long pieces = K / Vec16<XT>::kPerVec, blocks = 4ll * sms * (kQThreads / threads);
    if (K % Vec16<XT>::kPerVec == 0 && pieces > 0 && pieces <= static_cast<long long>(KEEP) * threads && M >= 2 * blocks)
        i8_quantize_rows_kernel<XT, KEEP><<<static_cast<unsigned>(blocks), threads, 0, s>>>(
            M, static_cast<int>(pieces), X, ldx, Q, ldq, scale);
    else
        i8_quantize_kernel<XT, true, KEEP><<<static_cast<unsigned>(M), threads, 0, s>>>(K, X, ldx, Q, ldq, scale);
    return cudaGetLastError();
}

template <int XT>
cudaError_t quantize_xt(long long M, long long K, const void *X, long long ldx, signed char *Q, long long ldq,
                        float *scale, int sms, cudaStream_t s) {
    const int es = static_cast<int>(sizeof(typename Elem<XT>::T));
    const bool vec = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && (M == 1 || ldx * es % 16 == 0) &&
                     (reinterpret_cast<uintptr_t>(Q) & 7u) == 0 && (M == 1 || ldq % 8 == 0);
    const unsigned grid = static_cast<unsigned>(M);
    if (!vec) {
        i8_quantize_kernel<XT, false, 1><<<grid, kQThreads, 0, s>>>(K, X, ldx, Q, ldq, scale);
        return cudaGetLastError();
    }
    // few pieces per thread while 256 threads hold the row, so that many rows are in flight per SM
    const long long pieces = K / Vec16<XT>::kPerVec;
    const int keep = pieces <= kQThreads ? 1 : pieces <= 2 * kQThreads ? 2 : pieces <= 4 * kQThreads ? 4 : 8;
    const long long want = (pieces + keep - 1) / keep;
    const int threads = want >= kQThreads ? kQThreads : static_cast<int>((want + 31) / 32 * 32 > 0 ? (want + 31) / 32 * 32 : 32);
    if (keep == 1) return quantize_keep<XT, 1>(M, threads, K, X, ldx, Q, ldq, scale, sms, s);
    if (keep == 2) return quantize_keep<XT, 2>(M, threads, K, X, ldx, Q, ldq, scale, sms, s);
    if (keep == 4) return quantize_keep<XT, 4>(M, threads, K, X, ldx, Q, ldq, scale, sms, s);
    return quantize_keep<XT, 8>(M, threads, K, X, ldx, Q, ldq, scale, sms, s);
}

}  // namespace

cudaError_t launch_i8_quantize(int x_dtype, long long M, long long K, const void *X, long long ldx, signed char *Q,
                               long long ldq, float *scale, int sms, cudaStream_t s) {
    if (x_dtype == kDtF32) return quantize_xt<kDtF32>(M, K, X, ldx, Q, ldq, scale, sms, s);
    if (x_dtype == kDtF16) return quantize_xt<kDtF16>(M, K, X, ldx, Q, ldq, scale, sms, s);
    if (x_dtype == kDtBF16) return quantize_xt<kDtBF16>(M, K, X, ldx, Q, ldq, scale, sms, s);
    return cudaErrorInvalidValue;
}

}  // namespace gb300
