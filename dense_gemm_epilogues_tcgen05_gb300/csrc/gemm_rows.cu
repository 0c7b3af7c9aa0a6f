// gemm_rows.cu -- the rows of a mixture of experts: the (token, expert) pairs
// sorted by expert, rows copied from token order into that order, the weighted
// sum back, and the gradients of both.
//
// A pair is p = t top + s (token t, slot s).  `row` holds each pair's place in
// expert order and `source` each place's pair; -1: none (a slot without an
// expert, a place behind the last pair).
//
// Measured (GB300): 16384 x 8 pairs over 256 experts sorted in 8.8 us (8.4 when the
// second kernel counted its own pairs before it waited, which nothing promises to
// work; over 1024 experts 41 and 38), 512 over 64 in 5.0 (the call's host side); 8 x
// 8192 rows of 4096 bf16 summed in 93 us, 6.5 TB/s; the gradients of that for 4099
// tokens of 2056, 6 slots, in 43 us, 4.8 TB/s (209 MB; 84 us with the loaded pieces
// unpacked at once, which left few of a thread's in flight; 51 with two blocks per SM,
// which spill nothing, instead of three; with a warp to a token and no barrier 55, and
// 4 % less only for 16384 tokens of 2048), 8192 tokens of 4096, 8 slots, in 190, 6.0
// TB/s.  What is on its way is held in registers; copies into shared memory, which need
// none, were not tried.
#include <algorithm>

#include "epilogue.cuh"
#include "kernel_args.h"
#include "launch.cuh"

namespace gb300 {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// ------------------------------------------------------------------ sorting --
// A counting sort in which nothing depends on the order of atomics: pairs of one
// expert stay in their order.  Many pairs: a first kernel counts each chunk's
// experts, the second gives every chunk its own place in each expert's range and
// its warps theirs, and each pair the number of equal ones before it in its warp
// (match).  Few pairs: the second kernel alone, one block.

constexpr int kCountThreads = 256;

__global__ void __launch_bounds__(kCountThreads) route_count_kernel(const __grid_constant__ RouteRowsArgs a) {
    extern __shared__ int counts[];
    begin_after();
    for (int e = threadIdx.x; e < a.E; e += kCountThreads) counts[e] = 0;
    __syncthreads();
    const int begin = blockIdx.x * a.chunk, end = min(begin + a.chunk, a.P);
    for (int p = begin + static_cast<int>(threadIdx.x); p < end; p += kCountThreads) {
        const int e = __ldg(a.expert + p);
        if (static_cast<unsigned>(e) < static_cast<unsigned>(a.E)) atomicAdd(&counts[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kCountThreads)
        a.counts[static_cast<long long>(e) * gridDim.x + blockIdx.x] = counts[e];
}

// The expert of this lane's pair p (-1: none, or the pair is not below `end`).
__device__ __forceinline__ int expert_of(const RouteRowsArgs &a, int p, int end) {
    const int e = p < end ? __ldg(a.expert + p) : -1;
    return static_cast<unsigned>(e) < static_cast<unsigned>(a.E) ? e : -1;
}

// Pairs begin .. end - 1 of one warp, 32 at a time: f(pair, expert, lanes of the same expert).  e_first, same_first: of
// the first 32.
template <typename F>
__device__ __forceinline__ void warp_pairs(const RouteRowsArgs &a, int begin, int end, int e_first, unsigned same_first,
                                           F f) {
    const int lane = threadIdx.x & 31;
    if (begin < end) f(begin + lane, e_first, same_first);
    for (int p0 = begin + 32; p0 < end; p0 += 32) {
        const int e = expert_of(a, p0 + lane, end);
        f(p0 + lane, e, __match_any_sync(kAll, e));
    }
}

__global__ void __launch_bounds__(1024) route_rows_kernel(const __grid_constant__ RouteRowsArgs a) {
    extern __shared__ int smem[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int *first = smem;              // E + 1: pairs of the experts before
    int *start = first + a.E + 1;   // E: an expert's pairs in the chunks before
    int *own = start + a.E;         // warps x E: counts, then places
    for (int i = threadIdx.x; i < warps * a.E; i += blockDim.x) own[i] = 0;
    if (threadIdx.x == 0) first[0] = 0;
    __syncthreads();
    begin_after();  // (for the pairs too: only who has waited is promised to see what earlier grids wrote)
    const int begin = blockIdx.x * a.chunk, end = min(begin + a.chunk, a.P);
    const int per = (a.chunk + warps * 32 - 1) / (warps * 32) * 32;  // pairs of a warp
    const int w0 = min(begin + warp * per, end), w1 = min(w0 + per, end);
    int *mine = own + warp * a.E;
    const int e_first = expert_of(a, w0 + lane, w1);  // on its way beside the counts
    // every expert's total, and what lies before this chunk (a warp takes an expert, its lanes the chunks)
    if (gridDim.x > 1) {
        const int chunks = gridDim.x;
        constexpr int kPer = (kRowsChunks + 31) / 32, kAtOnce = 8;  // loads of a lane per expert, experts at once
        for (int e0 = warp; e0 < a.E; e0 += kAtOnce * warps) {
            int n[kAtOnce][kPer];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    const int e = e0 + i * warps, c = lane + 32 * k;
                    n[i][k] = e < a.E && c < chunks ? __ldcg(a.counts + static_cast<long long>(e) * chunks + c) : 0;
                }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                int before = 0, total = 0;
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    before += lane + 32 * k < static_cast<int>(blockIdx.x) ? n[i][k] : 0;
                    total += n[i][k];
                }
                before = __reduce_add_sync(kAll, before);
                total = __reduce_add_sync(kAll, total);
                const int e = e0 + i * warps;
                if (lane == 0 && e < a.E) {
                    first[e + 1] = total;
                    start[e] = before;
                }
            }
        }
    }
    const unsigned same_first = __match_any_sync(kAll, e_first);
    warp_pairs(a, w0, w1, e_first, same_first, [&](int, int e, unsigned same) {
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    });
    __syncthreads();
    const auto sum_totals = [&] {  // by one warp: `first` from the experts' totals
        int base = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            int v = e < a.E ? first[e + 1] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(kAll, v, d);
                if (lane >= d) v += o;
            }
            if (e < a.E) first[e + 1] = base + v;
            base += __shfl_sync(kAll, v, 31);
        }
    };
    if (gridDim.x > 1 && warp == warps - 1) sum_totals();  // (while the others, if there are, place their warps)
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int at = gridDim.x > 1 ? start[e] : 0;
#pragma unroll 8
        for (int w = 0; w < warps; ++w) {
            const int n = own[w * a.E + e];
            own[w * a.E + e] = at;
            at += n;
        }
        if (gridDim.x == 1) first[e + 1] = at;
    }
    __syncthreads();
    if (gridDim.x == 1) {
        if (warp == 0) sum_totals();
        __syncthreads();
    }
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.offsets[e] = first[e];
    warp_pairs(a, w0, w1, e_first, same_first, [&](int p, int e, unsigned same) {
        int at = -1;
        if (e >= 0) {
            at = first[e] + mine[e] + __popc(same & ((1u << lane) - 1u));
            a.source[at] = p;
        }
        if (p < w1 && a.row != nullptr) a.row[p] = at;
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    });
    // the places behind the last pair
    for (int r = first[a.E] + static_cast<int>(blockIdx.x * blockDim.x + threadIdx.x); r < a.P;
         r += static_cast<int>(gridDim.x * blockDim.x))
        a.source[r] = -1;
}

// ----------------------------------------------------------------- movement --
// All three are bound by HBM; what they read and write, they do in 16-byte
// pieces where bases and pitches allow.  Sums run in fp32 in the order of the
// slots.

constexpr int kMoveThreads = 256;

// 16 bytes that are read once.
__device__ __forceinline__ uint4 ld_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// A piece of a row: 16 bytes (V) or one element, as stored until it is used, so that many are on their way at once.
template <int DT, bool V> struct Piece {
    static constexpr int N = Vec16<DT>::kPerVec;
    using Raw = uint4;
    static __device__ __forceinline__ Raw load(const void *row, long long i) { return ld_stream(static_cast<const uint4 *>(row) + i); }
    static __device__ __forceinline__ void unpack(const Raw &u, float (&f)[N]) { Vec16<DT>::unpack(u, f); }
    static __device__ __forceinline__ void store(void *row, long long i, const float (&f)[N]) {
        static_cast<uint4 *>(row)[i] = Vec16<DT>::pack(f);
    }
};
template <int DT> struct Piece<DT, false> {
    static constexpr int N = 1;
    using T = typename Elem<DT>::T;
    using Raw = T;
    static __device__ __forceinline__ Raw load(const void *row, long long i) { return static_cast<const T *>(row)[i]; }
    static __device__ __forceinline__ void unpack(const Raw &u, float (&f)[1]) { f[0] = Elem<DT>::load(&u); }
    static __device__ __forceinline__ void store(void *row, long long i, const float (&f)[1]) {
        static_cast<T *>(row)[i] = Elem<DT>::cvt(f[0]);
    }
};

template <int DT>
__device__ __forceinline__ const char *row_at(const void *base, long long row, long long ld) {
    return static_cast<const char *>(base) + row * ld * static_cast<long long>(sizeof(typename Elem<DT>::T));
}
template <int DT>
__device__ __forceinline__ char *row_at(void *base, long long row, long long ld) {
    return static_cast<char *>(base) + row * ld * static_cast<long long>(sizeof(typename Elem<DT>::T));
}

// A 16-byte piece of a row that is read again, and one that is written, with L2 eviction policies.
__device__ __forceinline__ uint4 ld_policy(const uint4 *p, uint64_t policy) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy));
    return v;
}
__device__ __forceinline__ void st_policy(uint4 *p, const uint4 &v, uint64_t policy) {
    asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w), "l"(policy)
                 : "memory");
}

// Pieces i, i + 32, ... below `pieces` of a row, times w, kAhead at once.  The rows written go first from L2, the
// tokens', which `top` rows are made of, last: 65536 rows of 4096 bf16 from 8192 tokens (537 MB written) 118 us, with
// neither policy 161, with the first alone 142.
template <int DT, bool V>
__device__ __forceinline__ void move_row(const void *x, void *y, int i, int pieces, bool scaled, float w) {
    using P = Piece<DT, V>;
    constexpr int kAhead = 8;
    const uint64_t keep = l2_policy_evict_last(), first = l2_policy_evict_first();
    for (; i < pieces; i += kAhead * 32) {
        typename P::Raw raw[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k * 32 < pieces) {
                if constexpr (V)
                    raw[k] = ld_policy(static_cast<const uint4 *>(x) + i + k * 32, keep);
                else
                    raw[k] = P::load(x, i + k * 32);
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i + k * 32 >= pieces) break;
            if (scaled) {
                float f[P::N];
                P::unpack(raw[k], f);
#pragma unroll
                for (int j = 0; j < P::N; ++j) f[j] *= w;
                if constexpr (V)
                    raw[k] = Vec16<DT>::pack(f);
                else
                    raw[k] = Elem<DT>::cvt(f[0]);
            }
            if constexpr (V)
                st_policy(static_cast<uint4 *>(y) + i + k * 32, raw[k], first);
            else
                static_cast<typename P::Raw *>(y)[i + k * 32] = raw[k];
        }
    }
}

// Y[r] = w[source[r]] X[source[r] / top]; places without a pair stay as they are.  A warp takes a part of a row of
// `part` pieces (all of it where there are rows for every warp), and the next one's pair while it does.
template <int DT, bool V>
__global__ void __launch_bounds__(kMoveThreads) rows_gather_kernel(const __grid_constant__ RowsArgs a) {
    begin_after();
    constexpr int N = Piece<DT, V>::N;
    const int lane = threadIdx.x & 31, whole = a.D / N;
    const long long step = static_cast<long long>(gridDim.x) * (kMoveThreads / 32), items = a.R * a.parts;
    const auto row_of = [&](long long i) { return a.parts == 1 ? i : static_cast<unsigned>(i) / static_cast<unsigned>(a.parts); };
    long long i = static_cast<long long>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5);
    int next = i < items ? __ldg(a.source + row_of(i)) : -1;
    for (; i < items; i += step) {
        const int p = next;
        next = i + step < items ? __ldg(a.source + row_of(i + step)) : -1;
        if (static_cast<unsigned>(p) >= static_cast<unsigned>(a.T) * static_cast<unsigned>(a.top)) continue;
        const bool scaled = a.weight != nullptr;
        const float w = scaled ? __ldg(a.weight + p) : 1.0f;
        const long long r = row_of(i);
        const int k = static_cast<int>(i - r * a.parts);
        const void *x = row_at<DT>(a.X, p / a.top, a.ldx);
        void *y = row_at<DT>(a.Y, r, a.ldy);
        move_row<DT, V>(x, y, k * a.part + lane, k + 1 < a.parts ? (k + 1) * a.part : whole, scaled, w);
        if (V && k + 1 == a.parts) move_row<DT, false>(x, y, whole * N + lane, a.D, scaled, w);
    }
}

constexpr int kSlots = 8;  // rows in flight per piece

// The rows and weights of kSlots slots of a token from slot s0 on; -1: none.
__device__ __forceinline__ void slots_of(const RowsArgs &a, long long t, int s0, int (&r)[kSlots], float (&w)[kSlots]) {
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
        r[s] = s0 + s < a.top ? __ldg(a.row + t * a.top + s0 + s) : -1;
        w[s] = a.weight != nullptr && s0 + s < a.top ? __ldg(a.weight + t * a.top + s0 + s) : 1.0f;
    }
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
        if (static_cast<unsigned>(r[s]) >= static_cast<unsigned>(a.R)) r[s] = -1;
}

// Piece i of Out[t] = sum_s w[t][s] Y[row[t][s]] + beta Out[t]; slots without a row add nothing.
// OUT: Out written as Y is read (else an element at a time).
template <int YT, int OT, bool V, bool OUT>
__device__ __forceinline__ void combine_piece(const RowsArgs &a, long long t, int i) {
    using P = Piece<YT, V>;
    using O = Piece<OT, OUT>;
    constexpr int OV = P::N / O::N;  // pieces of the output per piece of Y: 1, 2, N, or 0 for half a piece
    float acc[P::N];
    char *out = row_at<OT>(a.X, t, a.ldx) + static_cast<long long>(i) * P::N * sizeof(typename Elem<OT>::T);
#pragma unroll
    for (int j = 0; j < P::N; ++j) acc[j] = 0.0f;
    for (int s0 = 0; s0 < a.top; s0 += kSlots) {
        int r[kSlots];
        float w[kSlots];
        typename P::Raw raw[kSlots];
        slots_of(a, t, s0, r, w);
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            if (r[s] >= 0) raw[s] = P::load(row_at<YT>(a.Y, r[s], a.ldy), i);
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            if (r[s] >= 0) {
                float f[P::N];
                P::unpack(raw[s], f);
#pragma unroll
                for (int j = 0; j < P::N; ++j) acc[j] = fmaf(w[s], f[j], acc[j]);
            }
    }
    if constexpr (!OUT) {
        using T = typename Elem<OT>::T;
        T *o = reinterpret_cast<T *>(out);
#pragma unroll
        for (int j = 0; j < P::N; ++j) {
            if (a.beta != 0.0f) acc[j] = fmaf(a.beta, Elem<OT>::load(o + j), acc[j]);
            o[j] = Elem<OT>::cvt(acc[j]);
        }
    } else if constexpr (OV >= 1) {
#pragma unroll
        for (int v = 0; v < OV; ++v) {
            float o[O::N];
            if (a.beta != 0.0f) {
                Vec16<OT>::unpack(reinterpret_cast<const uint4 *>(out)[v], o);
#pragma unroll
                for (int j = 0; j < O::N; ++j) acc[v * O::N + j] = fmaf(a.beta, o[j], acc[v * O::N + j]);
            }
#pragma unroll
            for (int j = 0; j < O::N; ++j) o[j] = acc[v * O::N + j];
            O::store(out, v, o);
        }
    } else {  // fp32 rows to 16 bits: four values, 8 bytes
        using T = typename Elem<OT>::T;
        T *o = reinterpret_cast<T *>(out);
        if (a.beta != 0.0f) {
#pragma unroll
            for (int j = 0; j < P::N; ++j) acc[j] = fmaf(a.beta, Elem<OT>::load(o + j), acc[j]);
        }
        T four[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) four[j] = Elem<OT>::cvt(acc[j]);
        *reinterpret_cast<uint2 *>(o) = *reinterpret_cast<const uint2 *>(four);
    }
}

// V: Y may be read in 16-byte pieces, OUT: Out written so; REST: D is not of whole pieces (builds without it keep
// within their registers).
template <int YT, int OT, bool V, bool OUT, bool REST>
__global__ void __launch_bounds__(kMoveThreads, 4) rows_combine_kernel(const __grid_constant__ RowsArgs a) {
    begin_after();
    constexpr int N = Piece<YT, V>::N;
    const int whole = a.D / N, i = blockIdx.y * blockDim.x + threadIdx.x;
    if (i < whole)
        combine_piece<YT, OT, V, OUT>(a, blockIdx.x, i);
    else if (REST && i - whole < a.D - whole * N)  // an element a thread
        combine_piece<YT, OT, false, false>(a, blockIdx.x, whole * N + i - whole);
}

// Threads of a block: three blocks to an SM, or with an SM for every item one of three times the threads (64 tokens of
// 7168 fp32, 8 slots, 9.8 us instead of 12.6; 100 of 6931 bf16 14 instead of 25).
constexpr int kGradThreads = 320, kGradMost = 960;

// The sums over the warp of eight values of each lane: lane l (and those beside it) gets that of value l / 4.  Halves
// the values a lane carries with each exchange: 9 shuffles instead of 40.
__device__ __forceinline__ float warp_sums_of_8(const float (&v)[8]) {
    const int lane = threadIdx.x & 31;
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool hi = (lane & 16) != 0;
        a[i] = (hi ? v[i + 4] : v[i]) + __shfl_xor_sync(kAll, hi ? v[i] : v[i + 4], 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool hi = (lane & 8) != 0;
        b[i] = (hi ? a[i + 2] : a[i]) + __shfl_xor_sync(kAll, hi ? a[i] : a[i + 2], 8);
    }
    const bool hi = (lane & 4) != 0;
    float c = (hi ? b[1] : b[0]) + __shfl_xor_sync(kAll, hi ? b[0] : b[1], 4);
    c += __shfl_xor_sync(kAll, c, 2);
    return c + __shfl_xor_sync(kAll, c, 1);
}

// Step i of an item: dY[row] = w dOut[t] and what it adds to the dots dOut[t] . Y[row].
template <int DT, int YT, bool V>
__device__ __forceinline__ void grad_step(const RowsArgs &a, const void *d, const int *r, const float *w, int i,
                                          float (&dot)[kSlots]) {
    using P = Piece<DT, V>;
    using Q = Piece<YT, V>;
    // the wider piece of the two is the step: HV of P, YV of Q
    constexpr int N = P::N > Q::N ? P::N : Q::N, HV = N / P::N, YV = N / Q::N;
    float g[N];
#pragma unroll
    for (int v = 0; v < HV; ++v) {
        float h[P::N];
        P::unpack(P::load(d, static_cast<long long>(i) * HV + v), h);
#pragma unroll
        for (int j = 0; j < P::N; ++j) g[v * P::N + j] = h[j];
    }
#pragma unroll
    for (int v = 0; v < YV; ++v) {
        const long long at = static_cast<long long>(i) * YV + v;
        typename Q::Raw raw[kSlots];
        if (a.dweight != nullptr) {
#pragma unroll
            for (int s = 0; s < kSlots; ++s)
                if (r[s] >= 0) raw[s] = Q::load(row_at<YT>(a.Y, r[s], a.ldy), at);
        }
        if (a.dY != nullptr) {
#pragma unroll
            for (int s = 0; s < kSlots; ++s)
                if (r[s] >= 0) {
                    float o[Q::N];
#pragma unroll
                    for (int j = 0; j < Q::N; ++j) o[j] = w[s] * g[v * Q::N + j];
                    Q::store(row_at<YT>(a.dY, r[s], a.lddy), at, o);
                }
        }
        if (a.dweight != nullptr) {
#pragma unroll
            for (int s = 0; s < kSlots; ++s)
                if (r[s] >= 0) {
                    float y[Q::N];
                    Q::unpack(raw[s], y);
#pragma unroll
                    for (int j = 0; j < Q::N; ++j) dot[s] = fmaf(g[v * Q::N + j], y[j], dot[s]);
                }
        }
    }
}

// dY[row] = w dOut[t], dweight[t][s] = dOut[t] . Y[row]; slots without a row: dweight 0.  Persistent blocks; an item is
// a token and kSlots of its slots.  The next item's rows and weights are on their way while an item's rows are, and
// one barrier an item hands over both these and the partial sums.
template <int DT, int YT, bool V>
__global__ void __launch_bounds__(kGradMost, 1) rows_combine_grad_kernel(const __grid_constant__ RowsArgs a) {
    begin_after();
    constexpr int N = Piece<DT, V>::N > Piece<YT, V>::N ? Piece<DT, V>::N : Piece<YT, V>::N;
    __shared__ float part[2][kGradMost / 32][kSlots];
    __shared__ int rows[2][kSlots];  // (in shared memory: a thread's registers hold rows on their way)
    __shared__ float weights[2][kSlots];
    static_assert(kSlots == 8, "warp_sums_of_8");
    const int steps = a.D / N, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = blockDim.x;
    const int batches = (a.top + kSlots - 1) / kSlots;
    const int items = static_cast<int>(a.T) * batches;  // (at most 2^30)
    int next_row = -1;
    float next_weight = 1.0f;
    auto fetch = [&](int item) {  // by the first kSlots threads
        const int t = item / batches, s = (item - t * batches) * kSlots + tid;
        next_row = -1;
        next_weight = 1.0f;
        if (item < items && s < a.top) {
            const int r = __ldg(a.row + static_cast<long long>(t) * a.top + s);
            next_row = static_cast<unsigned>(r) < static_cast<unsigned>(a.R) ? r : -1;
            if (a.weight != nullptr) next_weight = __ldg(a.weight + static_cast<long long>(t) * a.top + s);
        }
    };
    if (tid < kSlots) {
        fetch(blockIdx.x);
        rows[0][tid] = next_row;
        weights[0][tid] = next_weight;
    }
    __syncthreads();
    int buf = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x, buf ^= 1) {
        const int t = item / batches, s0 = (item - t * batches) * kSlots;
        const void *d = row_at<DT>(a.X, t, a.ldx);
        const int *r = rows[buf];
        const float *w = weights[buf];
        float dot[kSlots];
#pragma unroll
        for (int s = 0; s < kSlots; ++s) dot[s] = 0.0f;
        if (tid < kSlots) fetch(item + static_cast<int>(gridDim.x));
        for (int i = tid; i < steps; i += n) grad_step<DT, YT, V>(a, d, r, w, i, dot);
        if (V && tid < a.D - steps * N) grad_step<DT, YT, false>(a, d, r, w, steps * N + tid, dot);
        const float sum = warp_sums_of_8(dot);
        if ((lane & 3) == 0) part[buf][warp][lane >> 2] = sum;
        if (tid < kSlots) {
            rows[buf ^ 1][tid] = next_row;
            weights[buf ^ 1][tid] = next_weight;
        }
        __syncthreads();
        if (a.dweight != nullptr && tid < kSlots && s0 + tid < a.top) {
            float v = 0.0f;
            for (int k = 0; k < n >> 5; ++k) v += part[buf][k][tid];
            a.dweight[static_cast<long long>(t) * a.top + s0 + tid] = v;
        }
    }
}

// Threads of a block, at most `most`, that share `pieces` of a row evenly: whole warps, no round nearly empty.
int block_for(int pieces, int most) {
    const int rounds = (pieces + most - 1) / most;
    return pieces <= 0 ? 32 : ((pieces + rounds - 1) / rounds + 31) / 32 * 32;
}

template <int YT, int OT>
cudaError_t launch_combine(const RowsArgs &a, bool vec, bool out_vec, cudaStream_t s) {
    const int per = vec ? Vec16<YT>::kPerVec : 1, pieces = a.D / per + a.D % per, n = block_for(pieces, kMoveThreads);
    const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>((pieces + n - 1) / n));
    const auto kern = !vec                          ? rows_combine_kernel<YT, OT, false, false, false>
                      : a.D % per == 0 && out_vec ? rows_combine_kernel<YT, OT, true, true, false>
                      : out_vec                   ? rows_combine_kernel<YT, OT, true, true, true>
                                                  : rows_combine_kernel<YT, OT, true, false, true>;
    return launch_after(kern, grid, n, 0, s, a);
}

template <int DT, int YT>
cudaError_t launch_grad(const RowsArgs &a, bool vec, int sms, cudaStream_t s) {
    const int per = vec ? (Vec16<DT>::kPerVec > Vec16<YT>::kPerVec ? Vec16<DT>::kPerVec : Vec16<YT>::kPerVec) : 1;
    const long long items = a.T * ((a.top + kSlots - 1) / kSlots);
    const int n = block_for(a.D / per, items <= sms ? kGradMost : kGradThreads);
    const long long most = static_cast<long long>(sms) * (n > kGradThreads ? 1 : 1024 / n);
    return launch_after(vec ? rows_combine_grad_kernel<DT, YT, true> : rows_combine_grad_kernel<DT, YT, false>,
                        dim3(static_cast<unsigned>(items < most ? items : most)), n, 0, s, a);
}

}  // namespace

cudaError_t launch_route_rows(const RouteRowsArgs &in, cudaStream_t s) {
    RouteRowsArgs a = in;
    const int chunks = route_rows_chunks(a.P);
    a.chunk = static_cast<int>(((static_cast<long long>(a.P) + chunks - 1) / chunks + 31) / 32 * 32);
    // as many warps as 32 KB of counts allow, and as there are pairs for
    const int most = 8192 / a.E < 32 ? 8192 / a.E : 32, want = (a.chunk + 31) / 32;
    const int warps = want < 1 ? 1 : want < most ? want : most, bytes = (2 * a.E + 1 + warps * a.E) * 4;
    if (chunks > 1) {
        cudaError_t err = launch_after(route_count_kernel, dim3(chunks), kCountThreads, a.E * 4, s, a);
        if (err != cudaSuccess) return err;
    }
    return launch_after(route_rows_kernel, dim3(chunks), 32 * warps, bytes, s, a);
}

// Few rows are split into parts, whole rounds of a warp, up to as many as 8 blocks per SM have warps: 8 rows of 6644
// bf16 in 4.7 us, 864 of 6931 fp32 with an odd pitch in 8.5; with a warp to a row 8.9 and 18.5.  (The single elements'
// kernels hold that many at a time; of the 16-byte pieces', whose registers are on their way, 3 run at once.)
cudaError_t launch_rows_gather(int dtype, const RowsArgs &in, bool vec, int sms, cudaStream_t s) {
    RowsArgs a = in;
    constexpr int kWarps = kMoveThreads / 32;
    const long long most = 8ll * sms;  // blocks
    const int pieces = vec ? a.D / (dtype == kDtF32 ? 4 : 8) : a.D, rounds = (pieces + 31) / 32;
    const long long parts = std::min<long long>(rounds, most * kWarps / a.R);
    a.part = parts > 1 ? static_cast<int>((rounds + parts - 1) / parts) * 32 : pieces;
    a.parts = parts > 1 ? (pieces + a.part - 1) / a.part : 1;
    const long long want = (a.R * a.parts + kWarps - 1) / kWarps;
    const unsigned grid = static_cast<unsigned>(want < most ? want : most);
    const auto launch = [&](auto whole, auto single) {
        return launch_after(vec ? whole : single, dim3(grid), kMoveThreads, 0, s, a);
    };
    if (dtype == kDtF32) return launch(rows_gather_kernel<kDtF32, true>, rows_gather_kernel<kDtF32, false>);
    if (dtype == kDtF16) return launch(rows_gather_kernel<kDtF16, true>, rows_gather_kernel<kDtF16, false>);
    if (dtype == kDtBF16) return launch(rows_gather_kernel<kDtBF16, true>, rows_gather_kernel<kDtBF16, false>);
    return cudaErrorInvalidValue;
}

cudaError_t launch_rows_combine(int y_dtype, int out_dtype, const RowsArgs &a, bool vec, bool out_vec, cudaStream_t s) {
    if (y_dtype == kDtF32 && out_dtype == kDtF32) return launch_combine<kDtF32, kDtF32>(a, vec, out_vec, s);
    if (y_dtype == kDtF32 && out_dtype == kDtF16) return launch_combine<kDtF32, kDtF16>(a, vec, out_vec, s);
    if (y_dtype == kDtF32 && out_dtype == kDtBF16) return launch_combine<kDtF32, kDtBF16>(a, vec, out_vec, s);
    if (y_dtype == kDtF16 && out_dtype == kDtF32) return launch_combine<kDtF16, kDtF32>(a, vec, out_vec, s);
    if (y_dtype == kDtF16 && out_dtype == kDtF16) return launch_combine<kDtF16, kDtF16>(a, vec, out_vec, s);
    if (y_dtype == kDtBF16 && out_dtype == kDtF32) return launch_combine<kDtBF16, kDtF32>(a, vec, out_vec, s);
    if (y_dtype == kDtBF16 && out_dtype == kDtBF16) return launch_combine<kDtBF16, kDtBF16>(a, vec, out_vec, s);
    return cudaErrorInvalidValue;
}

cudaError_t launch_rows_combine_grad(int d_dtype, int y_dtype, const RowsArgs &a, bool vec, int sms, cudaStream_t s) {
    if (d_dtype == kDtF32 && y_dtype == kDtF32) return launch_grad<kDtF32, kDtF32>(a, vec, sms, s);
    if (d_dtype == kDtF32 && y_dtype == kDtF16) return launch_grad<kDtF32, kDtF16>(a, vec, sms, s);
    if (d_dtype == kDtF32 && y_dtype == kDtBF16) return launch_grad<kDtF32, kDtBF16>(a, vec, sms, s);
    if (d_dtype == kDtF16 && y_dtype == kDtF16) return launch_grad<kDtF16, kDtF16>(a, vec, sms, s);
    if (d_dtype == kDtBF16 && y_dtype == kDtBF16) return launch_grad<kDtBF16, kDtBF16>(a, vec, sms, s);
    return cudaErrorInvalidValue;
}

}  // namespace gb300
