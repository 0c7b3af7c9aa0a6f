// gemm_route.cu -- a router's scores to each token's experts and weights, and
// the gradient of that.
//
//     s = softmax(x) or sigmoid(x),   sel = s + bias
//     groups: worth = the sum of a group's one or two highest sel; the best stay
//     the `top` highest sel of what stays, ties to the lower index
//     w = scale s, or scale s / (sum of the chosen s)
//
// A warp takes a token; lane l holds the experts l NPL .. l NPL + NPL - 1 in
// registers, so that lanes are in the experts' order and the experts of a group lie
// in neighbouring lanes.  A warp's maximum is one redux.  The top-th largest of the
// lanes' maxima bounds the chosen ones from below: what reaches it, rarely more than a
// few values over `top`, is gathered one to a lane (in the experts' order), and each
// counts those before it.
//
// Which experts are chosen is decided as by 64-bit scores.  Without a bias (and
// without sums over a group) the scores have the logits' order, and the logits
// are exact.  Otherwise fp32 scores decide wherever neighbours are further apart
// than their errors can be; else the token's scores are computed again in 64
// bits, of the candidates alone where that is enough (about one token in 1300 with
// 256 experts and sigmoid scores of ordinary spread; each of a token's in a lane of
// its own, since a 64-bit exponential takes a lane some microseconds).  Where most
// tokens' scores are close it is the whole time: 16384 tokens of 256 experts with one
// softmax logit 25 above the chosen ones 525 us, in groups of two 606; sigmoid logits
// around 17, 361 and 443; all logits equal, in groups, 444 (sigmoid) and 608.
//
// Bound by instructions (GB300: 900 per token of a warp, 16384 tokens to 8 of 256
// experts in 8 groups with a bias 18.4 to 19.2 us, without both 9.0; the logits' bytes
// would take 2.5): with a maximum of the warp per chosen expert 0.4 to 1.2 us more, with a
// search through a lane's registers in each round 43.  The gradient over 16384 x 128 softmax
// scores 6.4 us (bytes: 2.6).  One token: 5.6 us, the call's host side.
#include <cfloat>

#include "epilogue.cuh"
#include "kernel_args.h"
#include "launch.cuh"

namespace gb300 {

namespace {

constexpr int kRouteWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float warp_max(float v) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// -infinity and NaN: not available; +infinity counts as the largest finite
// value; -0 as 0, whose bits it must not be told from.
__device__ __forceinline__ float logit_value(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX) + 0.0f; }

// 1 / (1 + e^-x) by the hardware's 2^x and reciprocal; below 2^-126 it is 0.
__device__ __forceinline__ float sigmoid_approx(float x) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
}

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
    return warp_max(m);
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// Takes v into the larger two values seen.
template <typename F>
__device__ __forceinline__ void take_top2(F &t1, F &t2, F v) {
    const F low = t1 < v ? t1 : v;
    t1 = t1 < v ? v : t1;
    t2 = t2 < low ? low : t2;
}

// Whether this lane's group stays; lane g * per holds the worth of group g (-infinity: none), and the lanes beside it.
// Returns whether the lane has a group.
template <typename F>
__device__ __forceinline__ bool group_stays(F worth, int per, const RouteArgs &a, bool &kept) {
    const int lane = threadIdx.x & 31, g = lane / per;
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
        const F other = __shfl_sync(kAll, worth, h * per);
        rank += other > worth || (other == worth && h < g);
    }
    const bool is_group = g < a.groups && worth > -INFINITY;
    kept = is_group && rank < a.top_groups;
    return is_group;
}

// How far fp32 selection scores can be off: a difference of two by less than `score` + 2^-23 of the larger (0: exact).
// Whether x may in truth not be above y, the next one.
__device__ __forceinline__ bool too_close(float x, float y, float score) {
    return !(x - y > score + 0x1p-23f * fmaxf(fabsf(x), fabsf(y)));
}

// Sum of n over the lanes before this one.
__device__ __forceinline__ int lanes_before(int n) {
    int sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, sum, d);
        sum += (threadIdx.x & 31) >= static_cast<unsigned>(d) ? o : 0;
    }
    return sum - n;
}

struct Candidate {
    float value;
    int expert;
};

// The chosen experts of a token by fp32 values: lane s gets the s-th (or -1).  sel: the lane's selection scores,
// -infinity where there is none, no NaN; cand: 32 slots of the warp; margin: too_close's.  `exactly`(expert) is a
// selection score in 64 bits (warp-collective; -1: -infinity): it decides among the candidates where fp32 ones cannot.
// Returns whether even that is not enough (groups too close, or more candidates than lanes).
template <int NPL, typename Exactly>
__device__ __forceinline__ bool choose(const float (&sel)[NPL], const RouteArgs &a, float *stage, Candidate *cand,
                                       float margin, int &expert, Exactly exactly) {
    const int lane = threadIdx.x & 31;
    float val[NPL];  // -infinity: none, or struck out
#pragma unroll
    for (int j = 0; j < NPL; ++j) val[j] = sel[j];
    bool close = false;
    if (a.groups > 1) {
        // the worth of group g in lane g * per (and those beside it)
        const int per = a.group_lanes > 0 ? a.group_lanes : 1;
        float t1 = -INFINITY, t2 = -INFINITY;
        if (a.group_lanes > 0) {
#pragma unroll
            for (int j = 0; j < NPL; ++j) take_top2(t1, t2, sel[j]);
            for (int d = 1; d < per; d <<= 1) {
                const float o1 = __shfl_xor_sync(kAll, t1, d), o2 = __shfl_xor_sync(kAll, t2, d);
                take_top2(t1, t2, o1);
                t2 = fmaxf(t2, o2);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (lane * NPL + j < a.E) stage[lane * NPL + j] = sel[j];
            __syncwarp();
            if (lane < a.groups)
                for (int i = 0; i < a.group_size; ++i) {
                    const int at = i + lane < a.group_size ? i + lane : (i + lane) % a.group_size;  // (other banks)
                    take_top2(t1, t2, stage[lane * a.group_size + at]);
                }
            __syncwarp();
        }
        const float worth = t1 + (a.group_sum == 2 && t2 > -INFINITY ? t2 : 0.0f);
        bool kept;
        const int g = lane / per;
        const bool is_group = group_stays(worth, per, a, kept);
        if (margin > 0.0f) {
            const float low = -warp_max(kept ? -worth : -INFINITY), high = warp_max(is_group && !kept ? worth : -INFINITY);
            // (the biases' roundings go by the sums' terms, which may be far above the sums)
            const float size = warp_max(is_group ? fabsf(t1) + (t2 > -INFINITY ? fabsf(t2) : 0.0f) : 0.0f);
            if (high > -INFINITY) close = too_close(low, high, 2.0f * margin + 0x1p-22f * size);
        }
        unsigned stays = __ballot_sync(kAll, kept && lane == g * per);  // bit g * per
        if (close) {
            // The groups' worths in 64 bits, from the experts that may be among a group's highest: one to a lane.
            const float least = a.group_sum == 2 ? t2 : t1;
            if (lane == g * per && g < a.groups)
                cand[g].value = least > -INFINITY && least < INFINITY ? least - (margin + 0x1p-22f * fabsf(least)) : least;
            __syncwarp();
            unsigned flags = 0u;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                const int eg = a.group_lanes > 0 ? g : (lane * NPL + j) / a.group_size;
                if (val[j] > -INFINITY && val[j] >= cand[eg].value) flags |= 1u << j;
            }
            __syncwarp();
            if (__reduce_add_sync(kAll, __popc(flags)) > 32) return true;
            int at = lanes_before(__popc(flags));
            for (; flags != 0u; flags &= flags - 1u) cand[at++].expert = lane * NPL + __ffs(flags) - 1;
            const int total = __shfl_sync(kAll, at, 31);
            __syncwarp();
            const int e = lane < total ? cand[lane].expert : -1;
            __syncwarp();
            const double v = exactly(e);
            const int eg = e / a.group_size;
            double x1 = -INFINITY, x2 = -INFINITY;
            for (int i = 0; i < total; ++i) {
                const double o = __shfl_sync(kAll, v, i);
                if (__shfl_sync(kAll, eg, i) == lane) take_top2(x1, x2, o);
            }
            group_stays(x1 + (a.group_sum == 2 && x2 > -INFINITY ? x2 : 0.0), 1, a, kept);
            const unsigned by_group = __ballot_sync(kAll, kept);
            stays = __ballot_sync(kAll, lane == g * per && (by_group >> g & 1u) != 0u);
        }
        if (a.group_lanes > 0) {
            kept = (stays >> (g * per) & 1u) != 0u;
#pragma unroll
            for (int j = 0; j < NPL; ++j) val[j] = kept ? val[j] : -INFINITY;
        } else {
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                const int eg = (lane * NPL + j) / a.group_size;
                if (eg >= 32 || (stays >> eg & 1u) == 0) val[j] = -INFINITY;
            }
        }
    }
    const int rounds = margin > 0.0f ? a.top + 1 : a.top;  // one more than is chosen, to compare with
    float best = val[0], least = -INFINITY;
#pragma unroll
    for (int j = 1; j < NPL; ++j) best = fmaxf(best, val[j]);
    float rest = best;
    for (int s = 0; s < rounds; ++s) {
        least = warp_max(rest);
        rest = rest == least ? -INFINITY : rest;
    }
    // and what may in truth reach it
    if (margin > 0.0f && fabsf(least) < INFINITY) least -= margin + 0x1p-22f * fabsf(least);
    least = fmaxf(least, -FLT_MAX);
    int n = 0;
#pragma unroll
    for (int j = 0; j < NPL; ++j) n += val[j] >= least;
    const int total = __reduce_add_sync(kAll, n);
    expert = -1;
    if (total <= 32) {
        int at = lanes_before(n);
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (val[j] >= least) cand[at++] = {val[j], lane * NPL + j};
        __syncwarp();
        const bool candidate = lane < total;
        const float mine = candidate ? cand[lane].value : -INFINITY;
        const int my_expert = candidate ? cand[lane].expert : -1;
        __syncwarp();
        // each candidate's rank; the candidates are in the experts' order
        int rank = 0;
        for (int i = 0; i < total; i += 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float o = __shfl_sync(kAll, mine, i + k);
                rank += o > mine || (o == mine && i + k < lane);
            }
        }
        if (candidate) cand[rank] = {mine, my_expert};
        __syncwarp();
        const int found = min(rounds, total);
        const float value = lane < found ? cand[lane].value : 0.0f;
        expert = lane < min(found, a.top) ? cand[lane].expert : -1;
        __syncwarp();
        if (margin > 0.0f) {
            const float next = __shfl_down_sync(kAll, value, 1);
            if (__any_sync(kAll, lane + 1 < found && too_close(value, next, margin))) {
                const double v = exactly(my_expert);
                rank = 0;
                for (int i = 0; i < total; ++i) {
                    const double o = __shfl_sync(kAll, v, i);
                    rank += o > v || (o == v && i < lane);
                }
                if (candidate) cand[rank].expert = my_expert;
                __syncwarp();
                expert = lane < min(found, a.top) ? cand[lane].expert : -1;
                __syncwarp();
            }
        }
    } else {
        // many equal maxima, or more experts to choose than lanes can bound: through the registers
        float last = 0.0f;
        for (int found = 0; found < rounds; ++found) {
            const float top = warp_max(best);
            if (top == -INFINITY) break;
            if (margin > 0.0f && found > 0 && too_close(last, top, margin)) return true;
            last = top;
            if (found == a.top) break;
            const int owner = __ffs(__ballot_sync(kAll, best == top)) - 1;
            int j_top = 0;
            if (lane == owner) {
#pragma unroll
                for (int j = NPL - 1; j >= 0; --j) j_top = val[j] == top ? j : j_top;
                best = -INFINITY;
#pragma unroll
                for (int j = 0; j < NPL; ++j) {
                    if (j == j_top) val[j] = -INFINITY;
                    best = fmaxf(best, val[j]);
                }
            }
            const int e = owner * NPL + __shfl_sync(kAll, j_top, owner);
            if (lane == found) expert = e;
        }
    }
    return false;
}

// exp(x - m) of the lane's logits (0 for -infinity) and their sum over the warp.
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

// A selection score in 64 bits; m, sum: of the softmax.
__device__ __forceinline__ double exact_score(float x, float bias, int score, float m, double sum) {
    const double z = score == kScoreSoftmax ? exp(static_cast<double>(x) - static_cast<double>(m)) / sum
                                            : 1.0 / (1.0 + exp(-static_cast<double>(x)));
    return z + static_cast<double>(bias);
}
template <int LT>
__device__ __forceinline__ double exact_sum(const typename Elem<LT>::T *row, int E, float m) {
    double sum = 0.0;
#pragma unroll 4
    for (int e = threadIdx.x & 31; e < E; e += 32) {
        const float x = logit_value(Elem<LT>::load(row + e));
        sum += x > -INFINITY ? exp(static_cast<double>(x) - static_cast<double>(m)) : 0.0;
    }
    return warp_sum(sum);
}

// The choice by 64-bit scores, in `stage` (E values of the warp); few tokens come here.
template <int LT>
__device__ __noinline__ int choose_exactly(const typename Elem<LT>::T *row, float m, const RouteArgs &a, double *stage) {
    const int lane = threadIdx.x & 31;
    const double sum = a.score == kScoreSoftmax ? exact_sum<LT>(row, a.E, m) : 1.0;
#pragma unroll 4
    for (int e = lane; e < a.E; e += 32) {
        const float x = logit_value(Elem<LT>::load(row + e));
        const double v = exact_score(x, a.bias != nullptr ? __ldg(a.bias + e) : 0.0f, a.score, m, sum);
        stage[e] = x > -INFINITY && v > -INFINITY ? v : -INFINITY;
    }
    __syncwarp();
    if (a.groups > 1) {
        double t1 = -INFINITY, t2 = -INFINITY;
        if (lane < a.groups)
            for (int i = 0; i < a.group_size; ++i) take_top2(t1, t2, stage[lane * a.group_size + i]);
        bool kept;
        group_stays(t1 + (a.group_sum == 2 && t2 > -INFINITY ? t2 : 0.0), 1, a, kept);
        const unsigned stays = __ballot_sync(kAll, kept);
        for (int e = lane; e < a.E; e += 32)
            if ((stays >> (e / a.group_size) & 1u) == 0) stage[e] = -INFINITY;
        __syncwarp();
    }
    int expert = -1;
    for (int s = 0; s < a.top; ++s) {
        double best = -INFINITY;
        int at = a.E;
        for (int e = lane; e < a.E; e += 32) {
            const double v = stage[e];
            at = v > best ? e : at;
            best = v > best ? v : best;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const double o = __shfl_xor_sync(kAll, best, d);
            const int oe = __shfl_xor_sync(kAll, at, d);
            const bool takes = o > best || (o == best && oe < at);
            best = takes ? o : best;
            at = takes ? oe : at;
        }
        if (at >= a.E) break;
        if (lane == s) expert = at;
        if (lane == 0) stage[at] = -INFINITY;
        __syncwarp();
    }
    __syncwarp();
    return expert;
}

// The weight of this lane's chosen expert (lanes without one: 0).  m, sum: of the softmax over all experts, used
// where its scores are not renormalised.
__device__ __forceinline__ float chosen_score(float x, bool live, int score, bool renorm, float m, float sum,
                                              float &total) {
    float v;
    if (score == kScoreSoftmax) {
        if (renorm) m = warp_max(live ? x : -INFINITY);
        v = live && x > -INFINITY ? expf(x - m) : 0.0f;
        total = renorm ? warp_sum(v) : sum;
    } else {
        // s = e^min(x, 0) / (1 + e^-|x|).  Renormalised, the largest of the e^min(x, 0) is taken out, so that
        // scores below fp32's range keep their proportions.
        const float low = fminf(x, 0.0f);
        float c = 0.0f;
        if (renorm) {
            c = warp_max(live ? low : -INFINITY);
            c = c > -INFINITY ? c : 0.0f;
        }
        v = live && x > -INFINITY ? __fdiv_rn(expf(low - c), 1.0f + expf(-fabsf(x))) : 0.0f;
        total = renorm ? warp_sum(v) : 1.0f;
    }
    return v;
}

// BY_LOGIT: the selection scores have the logits' order.
template <int LT, int NPL, bool BY_LOGIT>
__global__ void __launch_bounds__(32 * kRouteWarps, NPL <= 8 ? 8 : 1) route_kernel(const __grid_constant__ RouteArgs a) {
    begin_after();
    using T = typename Elem<LT>::T;
    extern __shared__ double stage_all[];
    __shared__ Candidate cand_all[kRouteWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double *stage = stage_all + warp * a.stage;
    float b[BY_LOGIT ? 1 : NPL];
    if (!BY_LOGIT) {
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            const int e = lane * NPL + j;
            b[BY_LOGIT ? 0 : j] = a.bias != nullptr && e < a.E ? __ldg(a.bias + e) : 0.0f;
        }
    }
    for (long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + warp; t < a.T;
         t += static_cast<long long>(gridDim.x) * kRouteWarps) {
        const T *row = static_cast<const T *>(a.logits) + t * a.ldl;
        float x[NPL];
        load_logits<LT, NPL>(row, a.E, a.vec, x);
        float m = 0.0f, sum = 1.0f;
        int expert;
        if constexpr (BY_LOGIT) {
            if (a.score == kScoreSoftmax && !a.renorm) {
                float p[NPL];
                m = warp_max_of(x);
                sum = softmax_parts<NPL>(x, m, p);
            }
            choose<NPL>(x, a, reinterpret_cast<float *>(stage), cand_all[warp], 0.0f, expert, [](int) { return 0.0; });
        } else {
            float sel[NPL];
            if (a.score == kScoreSoftmax) {
                m = warp_max_of(x);
                sum = softmax_parts<NPL>(x, m, sel);
#pragma unroll
                for (int j = 0; j < NPL; ++j) sel[j] = __fdividef(sel[j], sum);
            } else {
#pragma unroll
                for (int j = 0; j < NPL; ++j) sel[j] = sigmoid_approx(x[j]);
            }
#pragma unroll
            for (int j = 0; j < NPL; ++j) sel[j] = x[j] > -INFINITY ? fmaxf(sel[j] + b[j], -INFINITY) : -INFINITY;  // (NaN: none)
            // What a difference of two scores may be off by, apart from the biases' roundings.  Sigmoid: each by less
            // than 1.6 x 2^-22, namely 1 for the quotient, 1/4 for the sum's rounding, 1/4 (the score's slope) for the
            // exponential and 0.09 for its argument's rounding (slope times |x| is at most 0.224).  Softmax, relative
            // to the largest score, 1 / sum: the sum's 37 roundings of 2^-24, common to both, and 9 each of
            // exponential and quotient.
            const float margin = a.score == kScoreSoftmax ? __fdividef(0x1p-18f, sum) : 0x1p-20f;
            const bool unsure = choose<NPL>(sel, a, reinterpret_cast<float *>(stage), cand_all[warp], margin, expert,
                                            [&](int e) {
                const double total = a.score == kScoreSoftmax ? exact_sum<LT>(row, a.E, m) : 1.0;  // (by the warp)
                return e < 0 ? -INFINITY : exact_score(logit_value(Elem<LT>::load(row + e)),
                                                       a.bias != nullptr ? __ldg(a.bias + e) : 0.0f, a.score, m, total);
            });
            if (unsure) expert = choose_exactly<LT>(row, m, a, stage);
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
//
// The order of experts does not matter here, so lanes take a row in pieces that
// lie beside each other.
// A row's elements over a warp: f(j, e) for this lane's j-th, expert e.  16-byte pieces (V) or single elements, each
// neighbouring lanes' (16384 tokens of 512 13 us, with NPL consecutive ones to a lane 20).
template <int PV, int NPL, typename F>
__device__ __forceinline__ void spread(bool v, F f) {
    const int lane = threadIdx.x & 31;
    if (NPL >= PV && v) {
#pragma unroll
        for (int j = 0; j < NPL; ++j) f(j, (j / PV * 32 + lane) * PV + j % PV);
    } else {
#pragma unroll
        for (int j = 0; j < NPL; ++j) f(j, j * 32 + lane);
    }
}

template <int LT, int NPL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_grad_kernel(const __grid_constant__ RouteGradArgs a) {
    begin_after();
    using T = typename Elem<LT>::T;
    constexpr int PV = Vec16<LT>::kPerVec;
    __shared__ __align__(16) float rows[kRouteWarps][32 * NPL];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *buf = rows[warp];
    const bool whole = a.score == kScoreSoftmax && !a.renorm;  // every logit has a gradient
    const long long step = static_cast<long long>(gridDim.x) * kRouteWarps;
    // Up to 256 experts the next token's arrays are on their way while a token is computed (65536 tokens of 256 29 us
    // instead of 32); with more, their registers cost more than that (16384 of 512 13.0, 14.1 with).
    constexpr bool kAhead = NPL <= 8;
    int next_expert = -1;
    float next_g = 0.0f, next_x[NPL];
    auto fetch = [&](long long t) {
        if (t >= a.T) return;
        next_expert = lane < a.top ? __ldg(a.expert + t * a.top + lane) : -1;
        next_g = lane < a.top ? __ldg(a.dweight + t * a.top + lane) : 0.0f;
        if (!whole) return;
        const T *row = static_cast<const T *>(a.logits) + t * a.ldl;
        if (NPL >= PV && a.vec) {
#pragma unroll
            for (int v = 0; v < NPL / PV; ++v) {
                const int e = (v * 32 + lane) * PV;
                if (e < a.E) {
                    Vec16<LT>::unpack(__ldg(reinterpret_cast<const uint4 *>(row + e)), &next_x[v * PV]);
                } else {
#pragma unroll
                    for (int j = 0; j < PV; ++j) next_x[v * PV + j] = -INFINITY;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NPL; ++j) next_x[j] = j * 32 + lane < a.E ? Elem<LT>::load(row + j * 32 + lane) : -INFINITY;
        }
    };
    long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + warp;
    if (kAhead) fetch(t);
    for (; t < a.T; t += step) {
        if (!kAhead) fetch(t);
        const bool live = next_expert >= 0 && next_expert < a.E;
        const int expert = live ? next_expert : -1;
        const float g = live ? a.scale * next_g : 0.0f;
        float d[NPL], m = 0.0f, sum = 1.0f, xs = 0.0f;
        if (whole) {
            float x[NPL];
#pragma unroll
            for (int j = 0; j < NPL; ++j) x[j] = logit_value(next_x[j]);
            if (kAhead) fetch(t + step);
            spread<PV, NPL>(a.vec, [&](int j, int e) { buf[e] = x[j]; });
            __syncwarp();
            if (live) xs = buf[expert];
            __syncwarp();
            m = warp_max_of(x);
            sum = softmax_parts<NPL>(x, m, d);
        } else {
            if (live) xs = logit_value(Elem<LT>::load(static_cast<const T *>(a.logits) + t * a.ldl + expert));
            if (kAhead) fetch(t + step);
        }
        float total;
        const float v = chosen_score(xs, live, a.score, a.renorm, m, sum, total);
        const float w = v > 0.0f ? __fdiv_rn(v, total) : 0.0f;
        // 1 - s of a sigmoid, without cancellation
        const float slope = a.score == kScoreSoftmax ? 1.0f
                                                     : __fdiv_rn(xs > 0.0f ? expf(-xs) : 1.0f, 1.0f + expf(-fabsf(xs)));
        const float mean = a.renorm || whole ? warp_sum(g * w) : 0.0f;
        const float c = slope * w * (a.renorm ? g - mean : g);
        const float share = sum > 0.0f ? -__fdiv_rn(mean, sum) : 0.0f;
#pragma unroll
        for (int j = 0; j < NPL; ++j) d[j] = whole ? d[j] * share : 0.0f;
        // The chosen experts' parts, added in the row's place in shared memory: by their lanes at once, or one after
        // the other where an expert is in two slots.
        spread<PV, NPL>(a.vec, [&](int j, int e) { buf[e] = d[j]; });
        __syncwarp();
        const unsigned same = __match_any_sync(kAll, expert);
        if (__any_sync(kAll, live && (same & (same - 1u)) != 0u)) {
            for (int s = 0; s < a.top; ++s) {
                if (lane == s && live) buf[expert] += c;
                __syncwarp();
            }
        } else if (live) {
            buf[expert] += c;
        }
        __syncwarp();
        spread<PV, NPL>(a.vec_out, [&](int j, int e) { d[j] = buf[e]; });
        __syncwarp();
        T *out = static_cast<T *>(a.dlogits) + t * a.ldd;
        if (NPL >= PV && a.vec_out) {
#pragma unroll
            for (int v4 = 0; v4 < NPL / PV; ++v4) {
                const int e = (v4 * 32 + lane) * PV;
                if (e < a.E) *reinterpret_cast<uint4 *>(out + e) = Vec16<LT>::pack(&d[v4 * PV]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (j * 32 + lane < a.E) out[j * 32 + lane] = Elem<LT>::cvt(d[j]);
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
    a.stage = !a.by_logit || (a.groups > 1 && a.group_lanes == 0) ? a.E : 0;
    const int bytes = kRouteWarps * a.stage * 8;
    return launch_after(a.by_logit ? route_kernel<LT, NPL, true> : route_kernel<LT, NPL, false>,
                        dim3(route_blocks(a.T, sms)), 32 * kRouteWarps, bytes, s, a);
}

template <int LT, int NPL>
cudaError_t launch_route_grad_npl(const RouteGradArgs &a, int sms, cudaStream_t s) {
    return launch_after(route_grad_kernel<LT, NPL>, dim3(route_blocks(a.T, sms)), 32 * kRouteWarps, 0, s, a);
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
