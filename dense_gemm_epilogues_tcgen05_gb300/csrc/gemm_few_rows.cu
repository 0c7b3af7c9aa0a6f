// gemm_few_rows.cu -- products for few rows (decoding), 16-bit values or 8-bit
// integers, dense or grouped: the weights stream once through shared memory and
// everything else hides behind that.
//
// One persistent block per SM walks tiles of 16 RG rows of W (output channels)
// by 8 NT rows of X of one group.  A producer thread keeps a ring of about
// 200 KB of TMA loads in flight across tiles -- a stage is KS boxes of 128 bytes
// of k of the W rows and of the X rows, one load each -- and in each of two teams,
// which take every other stage, warp (i, j) multiplies W row group i, box j; the
// partial sums of an output meet in shared memory at the end of a tile, in a
// fixed order.
//
// 16-bit values: mma.sync m16n8k16 with fp32 sums, joined every 512 k.  8-bit integers, up to four
// rows: dot products of four codes (dp4a); up to eight: mma.sync m16n8k32 on the
// codes; more: m16n8k16 on the codes expanded to binary16, fp32 sums moved into
// integers every 1024 k as in gemm_i8_tc.cu (the integer kind takes about 20
// clocks per SM for 16 x 8 x 32 on GB300, as long as HBM takes to bring its 512
// codes of W, so it does for eight rows and not for sixteen).  Integer sums are
// exact, so those results do not depend on the path.
//
// The sum over k does not care which k an MMA's slot holds as long as both
// operands agree, so lane (g, t) = (lane / 4, lane % 4) reads whole 16-byte units
// 2t and 2t + 1 of rows g and g + 8 of W and of rows g of X, and feeds their words
// to the MMAs in order.  Unit u of row r sits at u ^ (r % 8) (128-byte swizzle),
// which puts the eight units that a quarter-warp reads into different banks.
// Rows and k outside the matrices arrive as zeros; rows of X that belong to the
// next group are other columns of the MMA and are not stored.
//
// Bound: HBM, by the weights' bytes.  GB300: one row of 16384 x 16384 codes 46 us
// (5.9 TB/s), 16 rows 58 us, 64 experts x 64 rows 2048 x 4096 59 us (6.5 TB/s); two
// experts of 4096 x 4096 fp16, 4 rows, 13 us.  One load per stage and operand instead
// of four was worth 20 %: the issuing thread was the bound.  32 rows of 8-bit codes:
// 87 us, by their MMAs.
#include "grouped.cuh"

namespace gb300 {

namespace {

// Up to this many rows of X the products are dot products of four codes
// (dp4a); from the next on, MMAs.
constexpr int kGvDotRows = 4;

// RG * KS = 8 consumer warps.
template <int NT>
struct GvConfig {
    static constexpr int RG = NT <= 2 ? 2 : 4, KS = 8 / RG, TEAM = 8, TEAMS = 2, WARPS = TEAM * TEAMS;
    static constexpr int W_ROWS = 16 * RG, X_ROWS = 8 * NT;
    static constexpr int W_BOX = W_ROWS * 128, X_BOX = X_ROWS * 128;
    static constexpr int X_OFF = KS * W_BOX, STAGE_BYTES = KS * (W_BOX + X_BOX);
    static constexpr int BAR_BYTES = 256;
    static constexpr int PART_INTS = WARPS * 16 * X_ROWS;  // one 16 x X_ROWS block of sums per warp
    static constexpr int FIXED = 1024 + BAR_BYTES + 4 * PART_INTS + (group_table_bytes(kMaxGroups) + 15) / 16 * 16;
    static constexpr int FIT = (232448 - FIXED) / STAGE_BYTES, STAGES = FIT < 10 ? FIT & ~1 : 10;
    static constexpr int THREADS = 32 * (WARPS + 1);
    static constexpr int SMEM = FIXED + STAGES * STAGE_BYTES;
    static_assert(STAGES >= 4 && STAGES % TEAMS == 0 && 2 * STAGES * 8 + 16 <= BAR_BYTES, "a ring, and its barriers");
};

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int AB>
__device__ __forceinline__ void mma_16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    if constexpr (AB == kDtF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int dot16(const uint4 &a, const uint4 &b, int c) {
    c = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), c);
    c = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), c);
    c = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), c);
    return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), c);
}

struct GvTile {
    int g, n0, r0, nr;
};

__device__ __forceinline__ GvTile gv_tile(const GroupTable &t, long long tile, int tiles_n, int w_rows, int x_rows) {
    GvTile o;
    const int rt = static_cast<int>(tile / tiles_n);
    o.n0 = static_cast<int>(tile - static_cast<long long>(rt) * tiles_n) * w_rows;
    o.g = group_of(t, rt);
    o.r0 = t.lo[o.g] + (rt - t.first[o.g]) * x_rows;
    o.nr = min(x_rows, t.hi[o.g] - o.r0);
    return o;
}

template <int AB, int OUT, int NT>
__global__ void __launch_bounds__(GvConfig<NT>::THREADS, 1)
    few_rows_kernel(const __grid_constant__ GvMaps maps, const __grid_constant__ GroupedArgs a) {
    using Cfg = GvConfig<NT>;
    using OutT = typename Elem<OUT>::T;
    using SumT = typename SimtAcc<AB>::T;  // 32-bit integers or fp32
    constexpr int STAGES = Cfg::STAGES, KS = Cfg::KS, X_ROWS = Cfg::X_ROWS;
    constexpr int BOX_K = AB == kDtI8 ? 128 : 64;  // elements in 128 bytes
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + STAGES * Cfg::STAGE_BYTES);
    uint64_t *empty = full + STAGES;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(empty + STAGES);
    SumT *part = reinterpret_cast<SumT *>(reinterpret_cast<unsigned char *>(full) + Cfg::BAR_BYTES);
    int *table_mem = reinterpret_cast<int *>(part + Cfg::PART_INTS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], Cfg::TEAM);
        }
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&maps.w);
        tma_prefetch_desc(&maps.x);
    }
    grid_dep_wait();
    grid_dep_launch();
    const GroupTable t =
        group_table_build(table_mem, a.offsets, a.G, a.M, threadIdx.x, Cfg::THREADS, RowTilesOf{X_ROWS});
    const int tiles_n = (a.N + Cfg::W_ROWS - 1) / Cfg::W_ROWS;
    const long long tiles = static_cast<long long>(t.first[a.G]) * tiles_n;
    const int turns = (a.K + BOX_K * KS - 1) / (BOX_K * KS);  // stages per tile

    if (warp == Cfg::WARPS) {
        if (lane == 0) {
            // ----------------------------------------------------- producer --
            uint32_t stage = 0, phase = 0, armed = 0, armed_parity = 0;
            const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
            bool ok = true;
            for (long long tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
                const GvTile o = gv_tile(t, tile, tiles_n, Cfg::W_ROWS, X_ROWS);
                for (int i = 0; i < turns; ++i) {
                    if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, a.status)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[stage], Cfg::STAGE_BYTES);
                    armed |= 1u << stage;
                    armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                    unsigned char *st = smem + stage * Cfg::STAGE_BYTES;
                    if (a.K % BOX_K == 0 || (i + 1) * KS * BOX_K <= a.K) {
                        // whole boxes, those past K as zeros
                        tma_load_4d_hint(st, &maps.w, &full[stage], 0, o.n0, i * KS, o.g, once);
                        tma_load_4d_hint(st + Cfg::X_OFF, &maps.x, &full[stage], 0, o.r0, i * KS, 0, keep);
                    } else {
                        for (int j = 0; j < KS; ++j) {
                            const int k = (i * KS + j) * BOX_K;
                            tma_load_3d_hint(st + j * Cfg::W_BOX, &maps.w_tail, &full[stage], k, o.n0, o.g, once);
                            tma_load_3d_hint(st + Cfg::X_OFF + j * Cfg::X_BOX, &maps.x_tail, &full[stage], k, o.r0, 0,
                                             keep);
                        }
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (*abort_flag) {
                for (int s = 0; s < STAGES; ++s)
                    if (armed & (1u << s)) mbar_drain_wait(&full[s], (armed_parity >> s) & 1u, 100000000ull);
            }
        }
        return;
    }

    // ------------------------------------------------------------ consumers --
    // Team i takes every other stage; turns are numbered through all tiles.
    const int g8 = lane >> 2, t4 = lane & 3, team = warp / Cfg::TEAM, rg = warp % Cfg::TEAM / KS, ks = warp % KS;
    uint32_t stage = team, phase = 0;
    int first = team;  // this team's first turn of the tile
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const GvTile o = gv_tile(t, tile, tiles_n, Cfg::W_ROWS, X_ROWS);
        bool ok = true;
        auto turn = [&](auto &&multiply) {  // one stage: wait, this warp's units, release
            ok = mbar_wait_bounded(&full[stage], phase, abort_flag, a.status);
            if (!__all_sync(0xffffffffu, ok)) return false;
            const unsigned char *w = smem + stage * Cfg::STAGE_BYTES + ks * Cfg::W_BOX + (rg * 16 + g8) * 128;
            const unsigned char *x = smem + stage * Cfg::STAGE_BYTES + Cfg::X_OFF + ks * Cfg::X_BOX;
            uint4 p[2], q[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int at = ((2 * t4 + u) ^ g8) << 4;  // rows g8 and g8 + 8 have the same r % 8
                p[u] = *reinterpret_cast<const uint4 *>(w + at);
                q[u] = *reinterpret_cast<const uint4 *>(w + 8 * 128 + at);
            }
            multiply(p, q, x);
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
            if ((stage += Cfg::TEAMS) >= STAGES) {
                stage -= STAGES;
                phase ^= 1u;
            }
            return true;
        };
        if constexpr (AB != kDtI8) {
            // The MMA cuts off what falls below its fp32 sum's last place, always towards
            // zero, so every 512 k (8 stages of 64) that sum is added into another, rounded
            // to nearest, as in gemm_grouped_tc.cu.
            float sum[NT][4] = {}, d[NT][4] = {};
            int since = 0;
            for (int i = first; i < turns; i += Cfg::TEAMS) {
                const bool go = turn([&](const uint4 (&p)[2], const uint4 (&q)[2], const unsigned char *x) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(x + (n * 8 + g8) * 128 +
                                                                             (((2 * t4 + u) ^ g8) << 4));
                            mma_16<AB>(d[n], p[u].x, q[u].x, p[u].y, q[u].y, v.x, v.y);
                            mma_16<AB>(d[n], p[u].z, q[u].z, p[u].w, q[u].w, v.z, v.w);
                        }
                });
                if (!go) break;
                if ((++since & 7) == 0 || i + Cfg::TEAMS >= turns) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            sum[n][j] += d[n][j];
                            d[n][j] = 0.0f;
                        }
                }
            }
            // rows of W g8, g8 + 8; rows of X 2 t4, 2 t4 + 1 of each eight
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    part[(warp * X_ROWS + n * 8 + 2 * t4 + (i & 1)) * 16 + g8 + (i >> 1) * 8] = sum[n][i];
        } else if (NT == 1 && o.nr <= kGvDotRows) {
            int d[kGvDotRows][2] = {};
            for (int i = first; i < turns; i += Cfg::TEAMS) {
                const bool go = turn([&](const uint4 (&p)[2], const uint4 (&q)[2], const unsigned char *x) {
#pragma unroll
                    for (int r = 0; r < kGvDotRows; ++r) {
                        if (r >= o.nr) break;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(x + r * 128 + (((2 * t4 + u) ^ r) << 4));
                            d[r][0] = dot16(p[u], v, d[r][0]);
                            d[r][1] = dot16(q[u], v, d[r][1]);
                        }
                    }
                });
                if (!go) break;
            }
            // rows of W g8, g8 + 8, summed over the four lanes of each
#pragma unroll
            for (int r = 0; r < kGvDotRows; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    int v = d[r][i];
                    v += __shfl_xor_sync(0xffffffffu, v, 1);
                    v += __shfl_xor_sync(0xffffffffu, v, 2);
                    if (t4 == 0) part[(warp * X_ROWS + r) * 16 + g8 + i * 8] = v;
                }
        } else if constexpr (NT == 1) {
            int d[4] = {};
            for (int i = first; i < turns; i += Cfg::TEAMS) {
                const bool go = turn([&](const uint4 (&p)[2], const uint4 (&q)[2], const unsigned char *x) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(x + g8 * 128 + (((2 * t4 + u) ^ g8) << 4));
                        mma_s8(d, p[u].x, q[u].x, p[u].y, q[u].y, v.x, v.y);
                        mma_s8(d, p[u].z, q[u].z, p[u].w, q[u].w, v.z, v.w);
                    }
                });
                if (!go) break;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) part[(warp * X_ROWS + 2 * t4 + (i & 1)) * 16 + g8 + (i >> 1) * 8] = d[i];
        } else {
            int sum[NT][4] = {};
            float d[NT][4] = {};
            int since = 0;
            for (int i = first; i < turns; i += Cfg::TEAMS) {
                const bool go = turn([&](const uint4 (&p)[2], const uint4 (&q)[2], const unsigned char *x) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t pw[4] = {p[u].x, p[u].y, p[u].z, p[u].w};
                        const uint32_t qw[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
                        uint32_t pl[4], ph[4], ql[4], qh[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            expand4(pw[j], pl[j], ph[j]);
                            expand4(qw[j], ql[j], qh[j]);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(x + (n * 8 + g8) * 128 +
                                                                             (((2 * t4 + u) ^ g8) << 4));
                            const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t lo, hi;
                                expand4(vw[j], lo, hi);
                                mma_16<kDtF16>(d[n], pl[j], ql[j], ph[j], qh[j], lo, hi);
                            }
                        }
                    }
                });
                if (!go) break;
                if ((++since & 7) == 0 || i + Cfg::TEAMS >= turns) {  // 1024 k: the fp32 sums are exact so far
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            sum[n][j] += __float2int_rn(d[n][j]);
                            d[n][j] = 0.0f;
                        }
                }
            }
            // rows of W g8, g8 + 8; rows of X 2 t4, 2 t4 + 1 of each eight
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    part[(warp * X_ROWS + n * 8 + 2 * t4 + (i & 1)) * 16 + g8 + (i >> 1) * 8] = sum[n][i];
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * Cfg::WARPS) : "memory");
        for (int i = threadIdx.x; ok && i < Cfg::W_ROWS * X_ROWS; i += 32 * Cfg::WARPS) {
            const int r = i / Cfg::W_ROWS, in = i % Cfg::W_ROWS, n = o.n0 + in;
            if (r >= o.nr || n >= a.N) continue;
            SumT sum = 0;
#pragma unroll
            for (int j = 0; j < Cfg::TEAMS * KS; ++j)
                sum += part[((j / KS * Cfg::TEAM + (in >> 4) * KS + j % KS) * X_ROWS + r) * 16 + (in & 15)];
            const long long gn = static_cast<long long>(o.g) * a.N + n;
            const float s = product_factor(a.alpha, a.col_scale != nullptr ? a.col_scale + gn : nullptr,
                                           a.row_scale != nullptr ? a.row_scale + o.r0 + r : nullptr);
            OutT *c = static_cast<OutT *>(a.C) + (o.r0 + r) * a.ldc + n;
            const float bias = a.epilogue != kEpiNone ? a.bias[gn] : 0.0f;
            const float cin = a.beta != 0.0f ? Elem<OUT>::load(c) : 0.0f;
            *c = Elem<OUT>::cvt(grouped_value<OUT>(static_cast<float>(sum), s, a.beta, cin, bias, a.epilogue));
        }
        first = (first + turns) & 1;
        // The producer may give up between two consumers' looks at the flag: they leave together or not at all.
        if (barrier_any<1, 32 * Cfg::WARPS>(*abort_flag != 0)) break;
    }
}

template <int AB, int OUT, int NT>
cudaError_t launch_few_cfg(const GvMaps &maps, const GroupedArgs &a, int sms, cudaStream_t s) {
    using Cfg = GvConfig<NT>;
    auto kern = few_rows_kernel<AB, OUT, NT>;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
    if (err != cudaSuccess) return err;
    const long long row_tiles = a.M / Cfg::X_ROWS + (a.M < a.G ? a.M : a.G);
    const long long tiles = row_tiles * ((a.N + Cfg::W_ROWS - 1) / Cfg::W_ROWS);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles < sms ? tiles : sms), 1, 1);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

template <int AB, int OUT>
cudaError_t launch_few_nt(int nt, const GvMaps &maps, const GroupedArgs &a, int sms, cudaStream_t s) {
    if (nt == 1) return launch_few_cfg<AB, OUT, 1>(maps, a, sms, s);
    if (nt == 2) return launch_few_cfg<AB, OUT, 2>(maps, a, sms, s);
    if (nt == 4) return launch_few_cfg<AB, OUT, 4>(maps, a, sms, s);
    return cudaErrorInvalidValue;
}

template <int AB>
cudaError_t launch_few_out(int out, int nt, const GvMaps &maps, const GroupedArgs &a, int sms, cudaStream_t s) {
    if (out == kDtF32) return launch_few_nt<AB, kDtF32>(nt, maps, a, sms, s);
    if (out == kDtF16) return launch_few_nt<AB, kDtF16>(nt, maps, a, sms, s);
    if (out == kDtBF16) return launch_few_nt<AB, kDtBF16>(nt, maps, a, sms, s);
    return cudaErrorInvalidValue;
}

}  // namespace

int few_rows_w_rows(int nt) { return nt <= 2 ? GvConfig<1>::W_ROWS : GvConfig<4>::W_ROWS; }
int few_rows_boxes(int nt) { return nt <= 2 ? GvConfig<1>::KS : GvConfig<4>::KS; }

cudaError_t launch_few_rows(int ab, int out, int nt, const GvMaps &maps, const GroupedArgs &a, int sms,
                            cudaStream_t s) {
    if (ab == kDtI8) return launch_few_out<kDtI8>(out, nt, maps, a, sms, s);
    if (ab == kDtF16) return launch_few_out<kDtF16>(out, nt, maps, a, sms, s);
    if (ab == kDtBF16) return launch_few_out<kDtBF16>(out, nt, maps, a, sms, s);
    return cudaErrorInvalidValue;
}

}  // namespace gb300
