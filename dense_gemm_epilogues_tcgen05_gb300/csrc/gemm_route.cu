// gemm_route.cu -- a router's scores to each token's experts and weights, and
// the gradient of that.
//
//     s = softmax(x) or sigmoid(x),   sel = s + bias
//     groups: worth = the sum of a group's one or two highest sel; the best stay
//     the `top` highest sel of what stays, ties to the lower index
//     w = scale s, or scale s / (sum of the chosen s)
//
// A warp takes a token; lane l holds the experts l NPL .. l NPL + NPL - 1 in
// registers, so that the lowest lane of a ballot is the lowest expert, and the
// experts of a group lie in neighbouring lanes.  Each of the `top` rounds takes
// the maximum of the lanes' maxima (one redux on the value's bits, ordered as
// integers) and strikes it out.
//
// Which experts are chosen is decided as by 64-bit scores.  Without a bias (and
// without sums over a group) the scores have the logits' order, and the logits
// are exact.  Otherwise fp32 scores decide wherever neighbours are further apart
// than their errors can be; else the token's scores are computed again in 64
// bits (of 16384 tokens with 256 experts, about one in 300).
#include <cfloat>

#include "epilogue.cuh"
#include "kernel_args.h"

namespace gb300 {

namespace {

constexpr int kRouteWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

// Values as unsigned integers of the same order; 0 is below every value.
struct Order32 {
    using F = float;
    using K = unsigned;
    static __device__ __forceinline__ K key(F f) {
        const unsigned u = __float_as_uint(f);
        return u ^ (static_cast<unsigned>(static_cast<int>(u) >> 31) | 0x80000000u);
    }
    static __device__ __forceinline__ F value(K k) {
        return __uint_as_float(k ^ (static_cast<int>(k) < 0 ? 0x80000000u : kAll));
    }
    static __device__ __forceinline__ K warp_max(K k) { return __reduce_max_sync(kAll, k); }
};
struct Order64 {
    using F = double;
    using K = unsigned long long;
    static __device__ __forceinline__ K key(F f) {
        const long long u = __double_as_longlong(f);
        return static_cast<K>(u) ^ (static_cast<K>(u >> 63) | 0x8000000000000000ull);
    }
    static __device__ __forceinline__ K warp_max(K k) {
        const unsigned hi = __reduce_max_sync(kAll, static_cast<unsigned>(k >> 32));
        const unsigned lo = __reduce_max_sync(kAll, static_cast<unsigned>(k >> 32) == hi ? static_cast<unsigned>(k) : 0u);
        return static_cast<K>(hi) << 32 | lo;
    }
};

// -infinity and NaN: not available; +infinity counts as the largest finite
// value; -0 as 0, whose bits it must not be told from.
__device__ __forceinline__ float logit_value(float x) { return x > -INFINITY ? fminf(x, FLT_MAX) + 0.0f : -INFINITY; }

// This lane's logits of a row (-infinity past the last expert).
template <int LT, int NPL>
__device__ __forceinline__ void load_logits(const typename Elem<LT>::T *row, int E, bool vec, float (&x)[NPL]) {
    constexpr int PV = Vec16<LT>::kPerVec;
    const int e0 = (threadIdx.x & 31) * NPL;
    if (NPL >= PV && vec) {  // E is a multiple of PV then
#pragma unroll
        for (int v = 0; v < NPL / PV; ++v) {
            if (e0 + v * PV < E) {
                Vec16<LT>::unpack(__ldg(reinterpret_cast<const uint4 *>(row + e0) + v), &x[v * PV]);
            } else {
#pragma unroll
                for (int j = 0; j < PV; ++j) x[v * PV + j] = -INFINITY;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < NPL; ++j) x[j] = e0 + j < E ? Elem<LT>::load(row + e0 + j) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j) x[j] = logit_value(x[j]);
}

template <int NPL>
__device__ __forceinline__ float warp_max_of(const float (&x)[NPL]) {
    float m = x[0];
#pragma unroll
    for (int j = 1; j < NPL; ++j) m = fmaxf(m, x[j]);
    return Order32::value(Order32::warp_max(Order32::key(m)));
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// The larger two of two pairs.
template <typename F>
__device__ __forceinline__ void merge_top2(F &a1, F &a2, F b1, F b2) {
    const F low = a1 < b1 ? a1 : b1, second = a2 < b2 ? b2 : a2;
    a1 = a1 < b1 ? b1 : a1;
    a2 = low < second ? second : low;
}

// The chosen experts of a token: lane s gets the s-th (or -1).  sel: the lane's
// selection scores, -infinity where there is none.  Returns whether two values
// that the choice depends on are within margin (1 + their size) of each other.
template <class O, int NPL>
__device__ __forceinline__ bool choose(const typename O::F (&sel)[NPL], const RouteArgs &a, typename O::F *stage,
                                       float margin, int &expert) {
    using F = typename O::F;
    using K = typename O::K;
    const int lane = threadIdx.x & 31;
    K key[NPL];
#pragma unroll
    for (int j = 0; j < NPL; ++j) key[j] = sel[j] > -INFINITY ? O::key(sel[j]) : 0;
    bool close = false;
    if (a.groups > 1) {
        // the worth of group g in lane g * per (and those beside it)
        const int per = a.group_lanes > 0 ? a.group_lanes : 1;
        F t1 = -INFINITY, t2 = -INFINITY;
        if (a.group_lanes > 0) {
#pragma unroll
            for (int j = 0; j < NPL; ++j) merge_top2<F>(t1, t2, sel[j] > -INFINITY ? sel[j] : -INFINITY, -INFINITY);
            for (int d = 1; d < per; d <<= 1)
                merge_top2<F>(t1, t2, __shfl_xor_sync(kAll, t1, d), __shfl_xor_sync(kAll, t2, d));
        } else {
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (lane * NPL + j < a.E) stage[lane * NPL + j] = sel[j] > -INFINITY ? sel[j] : -INFINITY;
            __syncwarp();
            if (lane < a.groups)
                for (int i = 0; i < a.group_size; ++i) {
                    const int at = i + lane < a.group_size ? i + lane : (i + lane) % a.group_size;  // (other banks)
                    merge_top2<F>(t1, t2, stage[lane * a.group_size + at], -INFINITY);
                }
            __syncwarp();
        }
        const F worth = t1 + (a.group_sum == 2 && t2 > -INFINITY ? t2 : F(0));
        const int g = lane / per;
        int rank = 0;
        for (int h = 0; h < a.groups; ++h) {
            const F other = __shfl_sync(kAll, worth, h * per);
            rank += other > worth || (other == worth && h < g);
        }
        const bool is_group = g < a.groups && worth > -INFINITY, kept = is_group && rank < a.top_groups;
        if (margin > 0.0f) {
            const K none = ~K(0);
            const K low = ~O::warp_max(~(kept ? O::key(worth) : none)), high = O::warp_max(is_group && !kept ? O::key(worth) : 0);
            if (high != 0) {
                const float lo = Order32::value(static_cast<unsigned>(low)), hi = Order32::value(static_cast<unsigned>(high));
                close = !(lo - hi > 2.0f * margin * (1.0f + fmaxf(fabsf(lo), fabsf(hi))));
            }
        }
        const unsigned stays = __ballot_sync(kAll, kept);
        if (a.group_lanes > 0) {
#pragma unroll
            for (int j = 0; j < NPL; ++j) key[j] = kept ? key[j] : 0;
        } else {
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                const int eg = (lane * NPL + j) / a.group_size;
                if (eg >= 32 || (stays >> eg & 1u) == 0) key[j] = 0;
            }
        }
    }
    K best = key[0];
#pragma unroll
    for (int j = 1; j < NPL; ++j) best = best < key[j] ? key[j] : best;
    expert = -1;
    float last = 0.0f;
    const int rounds = margin > 0.0f ? a.top + 1 : a.top;
    for (int s = 0; s < rounds; ++s) {
        const K top = O::warp_max(best);
        if (top == 0) break;
        if (margin > 0.0f) {
            const float v = Order32::value(static_cast<unsigned>(top));
            if (s > 0) close = close || !(last - v > margin * (1.0f + fmaxf(fabsf(last), fabsf(v))));
            last = v;
            if (s == a.top) break;
        }
        const int owner = __ffs(__ballot_sync(kAll, best == top)) - 1;
        int j_top = 0;
        if (lane == owner) {
#pragma unroll
            for (int j = NPL - 1; j >= 0; --j) j_top = key[j] == top ? j : j_top;
            best = 0;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                if (j == j_top) key[j] = 0;
                best = best < key[j] ? key[j] : best;
            }
        }
        const int e = owner * NPL + __shfl_sync(kAll, j_top, owner);
        if (lane == s) expert = e;
    }
    return close;
}

// exp(x - m) of the lane's logits (0 for -infinity) and their sum over the warp.
template <typename F, int NPL>
__device__ __forceinline__ F softmax_parts(const float (&x)[NPL], float m, F (&p)[NPL]) {
    F sum = 0;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        p[j] = x[j] > -INFINITY ? exp(static_cast<F>(x[j]) - static_cast<F>(m)) : F(0);
        sum += p[j];
    }
    return warp_sum(sum);
}
template <int NPL>
__device__ __forceinline__ float softmax_parts(const float (&x)[NPL], float m, float (&p)[NPL]) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        p[j] = x[j] > -INFINITY ? expf(x[j] - m) : 0.0f;
        sum += p[j];
    }
    return warp_sum(sum);
}

template <int NPL>
__device__ __forceinline__ float bias_of(const RouteArgs &a, int j) {
    const int e = (threadIdx.x & 31) * NPL + j;
    return a.bias != nullptr && e < a.E ? __ldg(a.bias + e) : 0.0f;
}

// The choice by 64-bit scores.
template <int NPL>
__device__ __noinline__ int choose_exactly(const float (&x)[NPL], float m, const RouteArgs &a, double *stage) {
    double sel[NPL];
    if (a.score == kScoreSoftmax) {
        const double sum = softmax_parts<double, NPL>(x, m, sel);
#pragma unroll
        for (int j = 0; j < NPL; ++j) sel[j] /= sum;
    } else {
#pragma unroll
        for (int j = 0; j < NPL; ++j) sel[j] = 1.0 / (1.0 + exp(-static_cast<double>(x[j])));
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j) sel[j] = x[j] > -INFINITY ? sel[j] + static_cast<double>(bias_of<NPL>(a, j)) : -INFINITY;
    int expert;
    choose<Order64, NPL>(sel, a, stage, 0.0f, expert);
    return expert;
}

// The weight of this lane's chosen expert (lanes without one: 0).  m, sum: of the softmax over all experts, used
// where its scores are not renormalised.
__device__ __forceinline__ float chosen_score(float x, bool live, int score, bool renorm, float m, float sum,
                                              float &total) {
    float v;
    if (score == kScoreSoftmax) {
        if (renorm) m = Order32::value(Order32::warp_max(Order32::key(live ? x : -INFINITY)));
        v = live && x > -INFINITY ? expf(x - m) : 0.0f;
        total = renorm ? warp_sum(v) : sum;
    } else {
        // s = e^min(x, 0) / (1 + e^-|x|).  Renormalised, the largest of the e^min(x, 0) is taken out, so that
        // scores below fp32's range keep their proportions.
        const float low = fminf(x, 0.0f);
        float c = 0.0f;
        if (renorm) {
            c = Order32::value(Order32::warp_max(Order32::key(live ? low : -INFINITY)));
            c = c > -INFINITY ? c : 0.0f;
        }
        v = live && x > -INFINITY ? __fdiv_rn(expf(low - c), 1.0f + expf(-fabsf(x))) : 0.0f;
        total = renorm ? warp_sum(v) : 1.0f;
    }
    return v;
}

template <int LT, int NPL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const __grid_constant__ RouteArgs a) {
    using T = typename Elem<LT>::T;
    extern __shared__ double stage_all[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double *stage = stage_all + warp * a.stage;
    for (long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + warp; t < a.T;
         t += static_cast<long long>(gridDim.x) * kRouteWarps) {
        const T *row = static_cast<const T *>(a.logits) + t * a.ldl;
        float x[NPL];
        load_logits<LT, NPL>(row, a.E, a.vec, x);
        float m = 0.0f, sum = 1.0f;
        int expert;
        if (a.by_logit) {
            if (a.score == kScoreSoftmax && !a.renorm) {
                float p[NPL];
                m = warp_max_of(x);
                sum = softmax_parts<NPL>(x, m, p);
            }
            choose<Order32, NPL>(x, a, reinterpret_cast<float *>(stage), 0.0f, expert);
        } else {
            float sel[NPL];
            if (a.score == kScoreSoftmax) {
                m = warp_max_of(x);
                sum = softmax_parts<NPL>(x, m, sel);
#pragma unroll
                for (int j = 0; j < NPL; ++j) sel[j] = __fdividef(sel[j], sum);
            } else {
#pragma unroll
                for (int j = 0; j < NPL; ++j) sel[j] = __fdividef(1.0f, 1.0f + __expf(-x[j]));
            }
#pragma unroll
            for (int j = 0; j < NPL; ++j) sel[j] = x[j] > -INFINITY ? sel[j] + bias_of<NPL>(a, j) + 0.0f : -INFINITY;
            // What a difference of two scores may be off by, relative to 1 + the larger: sigmoid, two errors of
            // less than 2^-21 (exponential, quotient, the bias's addition); softmax, its sum's 37 roundings too.
            const float margin = a.score == kScoreSoftmax ? 0x1p-17f : 0x1p-19f;
            if (choose<Order32, NPL>(sel, a, reinterpret_cast<float *>(stage), margin, expert)) {
                float copy[NPL];  // (the call takes an address: x itself stays in registers)
#pragma unroll
                for (int j = 0; j < NPL; ++j) copy[j] = x[j];
                expert = choose_exactly<NPL>(copy, m, a, stage);
            }
        }
        const bool live = expert >= 0;
        const float xs = live ? logit_value(Elem<LT>::load(row + expert)) : 0.0f;
        float total;
        const float v = chosen_score(xs, live, a.score, a.renorm, m, sum, total);
        if (lane < a.top) {
            a.expert[t * a.top + lane] = expert;
            a.weight[t * a.top + lane] = v > 0.0f ? a.scale * __fdiv_rn(v, total) : 0.0f;
        }
    }
}

// With w = v / total the weight before `scale`, g = scale * dweight and d the
// derivative of a chosen score by its logit over the score (softmax 1, sigmoid
// 1 - s):
//     renormalised   dx_j += d_j w_j (g_j - sum_i g_i w_i)
//     sigmoid        dx_j += g_j s_j (1 - s_j)
//     softmax        dx_j += g_j p_j, and every expert's dx_e -= p_e sum_i g_i p_i
template <int LT, int NPL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_grad_kernel(const __grid_constant__ RouteGradArgs a) {
    using T = typename Elem<LT>::T;
    constexpr int PV = Vec16<LT>::kPerVec;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool whole = a.score == kScoreSoftmax && !a.renorm;  // every logit has a gradient
    for (long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + warp; t < a.T;
         t += static_cast<long long>(gridDim.x) * kRouteWarps) {
        const T *row = static_cast<const T *>(a.logits) + t * a.ldl;
        int expert = lane < a.top ? a.expert[t * a.top + lane] : -1;
        const bool live = expert >= 0 && expert < a.E;
        expert = live ? expert : -1;
        const float g = live ? a.scale * a.dweight[t * a.top + lane] : 0.0f;
        const float xs = live ? logit_value(Elem<LT>::load(row + expert)) : 0.0f;
        float d[NPL], m = 0.0f, sum = 1.0f;
        if (whole) {
            float x[NPL];
            load_logits<LT, NPL>(row, a.E, a.vec, x);
            m = warp_max_of(x);
            sum = softmax_parts<NPL>(x, m, d);
            const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
#pragma unroll
            for (int j = 0; j < NPL; ++j) d[j] *= inv;
        }
        float total;
        const float v = chosen_score(xs, live, a.score, a.renorm, m, sum, total);
        const float w = v > 0.0f ? __fdiv_rn(v, total) : 0.0f;
        // 1 - s of a sigmoid, without cancellation
        const float slope = a.score == kScoreSoftmax ? 1.0f
                                                     : __fdiv_rn(xs > 0.0f ? expf(-xs) : 1.0f, 1.0f + expf(-fabsf(xs)));
        const float mean = a.renorm || whole ? warp_sum(g * w) : 0.0f;
        const float c = slope * w * (a.renorm ? g - mean : g);
        if (whole) {
#pragma unroll
            for (int j = 0; j < NPL; ++j) d[j] = -d[j] * mean;
        } else {
#pragma unroll
            for (int j = 0; j < NPL; ++j) d[j] = 0.0f;
        }
        for (int s = 0; s < a.top; ++s) {  // in the slots' order, also where an expert is in two of them
            const int e = __shfl_sync(kAll, expert, s) - lane * NPL;
            const float cs = __shfl_sync(kAll, c, s);
#pragma unroll
            for (int j = 0; j < NPL; ++j) d[j] += e == j ? cs : 0.0f;
        }
        T *out = static_cast<T *>(a.dlogits) + t * a.ldd;
        const int e0 = lane * NPL;
        if (NPL >= PV && a.vec_out) {
#pragma unroll
            for (int v4 = 0; v4 < NPL / PV; ++v4)
                if (e0 + v4 * PV < a.E) reinterpret_cast<uint4 *>(out + e0)[v4] = Vec16<LT>::pack(&d[v4 * PV]);
        } else {
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (e0 + j < a.E) out[e0 + j] = Elem<LT>::cvt(d[j]);
        }
    }
}

int route_blocks(long long T, int sms) {
    const long long want = (T + kRouteWarps - 1) / kRouteWarps, most = 16ll * sms;
    return static_cast<int>(want < most ? want : most);
}

template <int LT, int NPL>
cudaError_t launch_route_npl(const RouteArgs &in, int sms, cudaStream_t s) {
    RouteArgs a = in;
    a.group_size = a.E / a.groups;
    a.group_lanes = 0;
    if (a.groups > 1 && a.E == 32 * NPL && 32 % a.groups == 0) a.group_lanes = 32 / a.groups;
    a.stage = a.groups > 1 && a.group_lanes == 0 ? a.E : 0;
    route_kernel<LT, NPL><<<route_blocks(a.T, sms), 32 * kRouteWarps, kRouteWarps * a.stage * 8, s>>>(a);
    return cudaGetLastError();
}

template <int LT, int NPL>
cudaError_t launch_route_grad_npl(const RouteGradArgs &a, int sms, cudaStream_t s) {
    route_grad_kernel<LT, NPL><<<route_blocks(a.T, sms), 32 * kRouteWarps, 0, s>>>(a);
    return cudaGetLastError();
}

template <int LT>
cudaError_t launch_route_lt(const RouteArgs &a, int sms, cudaStream_t s) {
    if (a.E <= 32) return launch_route_npl<LT, 1>(a, sms, s);
    if (a.E <= 64) return launch_route_npl<LT, 2>(a, sms, s);
    if (a.E <= 128) return launch_route_npl<LT, 4>(a, sms, s);
    if (a.E <= 256) return launch_route_npl<LT, 8>(a, sms, s);
    if (a.E <= 512) return launch_route_npl<LT, 16>(a, sms, s);
    return launch_route_npl<LT, 32>(a, sms, s);
}

template <int LT>
cudaError_t launch_route_grad_lt(const RouteGradArgs &a, int sms, cudaStream_t s) {
    if (a.E <= 32) return launch_route_grad_npl<LT, 1>(a, sms, s);
    if (a.E <= 64) return launch_route_grad_npl<LT, 2>(a, sms, s);
    if (a.E <= 128) return launch_route_grad_npl<LT, 4>(a, sms, s);
    if (a.E <= 256) return launch_route_grad_npl<LT, 8>(a, sms, s);
    if (a.E <= 512) return launch_route_grad_npl<LT, 16>(a, sms, s);
    return launch_route_grad_npl<LT, 32>(a, sms, s);
}

}  // namespace

cudaError_t launch_route(int l_dtype, const RouteArgs &a, int sms, cudaStream_t s) {
    if (l_dtype == kDtF32) return launch_route_lt<kDtF32>(a, sms, s);
    if (l_dtype == kDtF16) return launch_route_lt<kDtF16>(a, sms, s);
    if (l_dtype == kDtBF16) return launch_route_lt<kDtBF16>(a, sms, s);
    return cudaErrorInvalidValue;
}

cudaError_t launch_route_grad(int l_dtype, const RouteGradArgs &a, int sms, cudaStream_t s) {
    if (l_dtype == kDtF32) return launch_route_grad_lt<kDtF32>(a, sms, s);
    if (l_dtype == kDtF16) return launch_route_grad_lt<kDtF16>(a, sms, s);
    if (l_dtype == kDtBF16) return launch_route_grad_lt<kDtBF16>(a, sms, s);
    return cudaErrorInvalidValue;
}

}  // namespace gb300
