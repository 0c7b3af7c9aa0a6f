// gemm_i8_tc.cu -- 8-bit integer products on the tensor cores, dense (one
// group) or grouped by expert:
//
//     C[r][f] = act(alpha xs[r] ws[g][f] sum_k X[r][k] W[g][f][k] + beta C[r][f] + bias[g][f])
//
// sm_103a's tensor cores have no fast integer kind, but every 8-bit integer is
// a binary16 number and so is every product's value in the fp32 accumulator's
// 24 bits: 1024 products of at most 128 * 128 sum to at most 2^24.  So the
// codes are expanded to binary16 on the way to the MMA (kind::f16, the bf16
// rate), and every 1024 k the epilogue warps take the fp32 accumulator --
// exact so far -- into 32-bit integers in registers, while the MMA fills the
// other accumulator.  The integer sum is exact for any K the interface allows,
// whatever the codes.
//
// The product is computed transposed on SM pairs, as in gemm_grouped_tc.cu: W's
// 256 rows are the MMA's rows, up to 192 rows of X its columns.  Per CTA:
//
//   warp 0        TMA producer: 128 rows of W and half of the tile's rows of X,
//                 128 k (bytes) deep, into a ring of 28 KB stages of codes (as many as fit),
//                 on this CTA's own barriers;
//   warp 1        MMA issuer (leader CTA only);
//   warps 4-19    converters, four sets of four; a set takes one 64-k half of
//                 every other stage.  A thread expands one row of W into tensor
//                 memory (the MMA's first operand: 32 columns of two values, so
//                 expanded W never crosses shared memory), and a warp one
//                 16-byte column of each row of X into a swizzled 16-bit tile;
//                 four to ten slots of each;
//   warps 20-27   epilogue: two per 32-lane quadrant, half of the columns each;
//                 96 integer sums per thread, then as in gemm_grouped_tc.cu.
//
// A code becomes binary16 by a byte permute into the mantissa of 1024 (the sign
// bit flipped first: 1024 + 128 + code) and one subtraction of 1152: five
// instructions for four codes, all exact.
//
// Registers: 28 warps launch with 72 each; the warpgroups then trade them (32
// for the issuers, 48 for each converter set, 136 for each epilogue set: 496 of
// the 504 that seven warps of a sub-partition launched with).
//
// Bound and measured (GB300, 8192 x 4096 x 4096 codes, bias and GELU, bf16 out):
// 212 us, 1.30 PFLOP/s.  The tensor pipe is busy 50 % and the issue slots 52 % of
// the time, so neither is the bound; no counter names the latency that is.  Shared memory would allow 1.08 of the MMAs'
// time at 192 columns: per 128 k a CTA moves 32 KB of W and 768 bytes per row of X
// against the MMA's 8 clocks per row.  On the way: arrives with release at cluster
// scope 372 us, fences restricted to shared memory 241 us; outputs of one accumulator
// straight from fp32 228 -> 217 us; outputs stored from registers and one more stage
// of codes 217 -> 210 us; the fence behind the warp's meeting 210 -> 212 us (other boxes).
#include <algorithm>

#include "gemm_tcgen05.cuh"
#include "grouped.cuh"

namespace gb300 {

namespace {

struct I8Config {
    static constexpr int BK = 128, MAX_STAGES = 8, MAX_SLOTS = 12;
    static constexpr int W_BYTES = 128 * BK;
    static constexpr int CHUNK_HALVES = 1024 / 64;  // 64-k halves summed in fp32
    static constexpr int W_SLOT_COLS = 32, TMEM_COLS = 512;
    static constexpr int SETS = 4;                  // converter sets of four warps
    static constexpr int CONV_WARP0 = 4, EPI_WARP0 = CONV_WARP0 + 4 * SETS, THREADS = 32 * (EPI_WARP0 + 8);
    // registers per thread: at launch, then the issuers', the converters', the epilogue's
    static constexpr int LAUNCH_REGS = 72, ISSUE_REGS = 32, CONV_REGS = 48, EPI_REGS = 136;
    static_assert(ISSUE_REGS + SETS * CONV_REGS + 2 * EPI_REGS <= (SETS + 3) * LAUNCH_REGS, "the trade adds up");
    static constexpr int BAR_BYTES = 512, SMEM_MAX = 232448;
    static_assert((2 * MAX_STAGES + 2 * MAX_SLOTS + 5) * 8 + 8 <= BAR_BYTES, "barriers fit their slot");
    // after up to 1023 bytes of alignment: [stages][slots][barriers][group table]
    static int fixed_bytes(int G) { return 1024 + BAR_BYTES + (group_table_bytes(G) + 15) / 16 * 16; }
};

// What follows from the widest row tile `most` and the group count: most / 2
// rows of X per CTA; tensor memory beside the two accumulators holds slots of
// expanded W, with as many of X in shared memory; the rest of shared memory
// holds stages of codes.
struct I8Shape {
    int stage_bytes, slot_bytes, slots, stages;
    __host__ __device__ I8Shape(int most, int stages_) : stages(stages_) {
        stage_bytes = I8Config::W_BYTES + most / 2 * I8Config::BK;
        slot_bytes = most / 2 * 128;  // 64 k in 16 bits
        const int cols = (I8Config::TMEM_COLS - 2 * most) / I8Config::W_SLOT_COLS;
        // Two sets can skip uses of a stage and of a slot, and a parity wait is
        // only right within one use.  A set at half h has had half h - 4 accepted,
        // so the issuer has consumed every half up to h - 4 - slots: that covers
        // the slot's use before the last (slots >= 4) and the stage's use before
        // this one (2 stages >= slots + 5).
        slots = cols < I8Config::MAX_SLOTS ? cols : I8Config::MAX_SLOTS;
        if (slots > 2 * stages - 5) slots = 2 * stages - 5;
        slots &= ~1;  // a stage's two halves are announced together
    }
    int bytes() const { return slots * slot_bytes + stages * stage_bytes; }
};

template <int OUT>
__global__ void __launch_bounds__(I8Config::THREADS, 1)
    i8_tc_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX32,
                 const __grid_constant__ CUtensorMap tmX16, const __grid_constant__ GtcArgs args) {
    using Cfg = I8Config;
    constexpr int CL = 2;
    const I8Shape sh(args.most, args.stages);
    const uint32_t slots = sh.slots, stages = sh.stages;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char *slot_base = smem + stages * sh.stage_bytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(slot_base + slots * sh.slot_bytes);  // codes landed
    uint64_t *empty = full + Cfg::MAX_STAGES;   // codes read by both converter sets
    uint64_t *ready = empty + Cfg::MAX_STAGES;  // (leader's) two slots, one stage, expanded in both CTAs
    uint64_t *freed = ready + Cfg::MAX_SLOTS;   // a slot read by the MMA
    uint64_t *tfull = freed + Cfg::MAX_SLOTS;
    uint64_t *tempty = tfull + 2;
    uint64_t *mma_done = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();  // 0: leader
    const int cluster = blockIdx.x / CL, nclusters = gridDim.x / CL;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::MAX_STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 8);
        }
        for (int s = 0; s < Cfg::MAX_SLOTS; ++s) {
            mbar_init(&ready[s], CL * 8);
            mbar_init(&freed[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], CL * 8);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX32);
        tma_prefetch_desc(&tmX16);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish_pair();
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    grid_dep_wait();
    grid_dep_launch();
    const GroupTable table = group_table_build(reinterpret_cast<int *>(reinterpret_cast<unsigned char *>(full) + Cfg::BAR_BYTES), args.offsets, args.G,
                                               args.T, threadIdx.x, Cfg::THREADS, RowTilesOf{args.most});
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t ready0_leader = mapa_shared(smem_u32(&ready[0]), 0);
    const uint32_t acc_stride = args.most, w_slot0 = tmem_base + 2 * acc_stride;
    const uint32_t tempty0_leader = mapa_shared(smem_u32(&tempty[0]), 0);
    const uint32_t abort_local = smem_u32(const_cast<int *>(abort_flag));
    const long long tiles = static_cast<long long>(table.first[args.G]) * args.tiles_f;
    const int num_kb = (args.K + Cfg::BK - 1) / Cfg::BK;

    if (warp < Cfg::CONV_WARP0) {
        regs_decrease<Cfg::ISSUE_REGS>();
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ TMA producer --
            uint32_t stage = 0, phase = 0;
            bool ok = true, issued = false;
            const uint64_t keep = l2_policy_evict_last();
            for (long long tile = cluster; ok && tile < tiles; tile += nclusters) {
                const GroupedTile t = row_tile(table, tile, args.tiles_f, args.K);
                const int f = t.f0 + static_cast<int>(rank) * 128, bnh = t.bn >> 1;
                const int r0 = t.r0 + static_cast<int>(rank) * bnh;
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!pair_wait<CL>(&empty[stage], phase ^ 1u, abort_flag, args.status, abort_local, rank)) {
                        ok = false;
                        break;
                    }
                    issued = true;
                    unsigned char *sW = smem + stage * sh.stage_bytes, *sX = sW + Cfg::W_BYTES;
                    const int k = kb * Cfg::BK;
                    mbar_arrive_expect_tx(&full[stage], Cfg::W_BYTES + bnh * 128);
                    tma_load_3d_hint(sW, &tmW, &full[stage], k, f, t.g, keep);
                    int r = 0;
                    for (; r + 32 <= bnh; r += 32)
                        tma_load_3d_hint(sX + r * 128, &tmX32, &full[stage], k, r0 + r, 0, keep);
                    for (; r < bnh; r += 16)
                        tma_load_3d_hint(sX + r * 128, &tmX16, &full[stage], k, r0 + r, 0, keep);
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (*abort_flag && issued) {
                // Unwinding: loads in flight complete within microseconds; give
                // them time to land before this CTA's shared memory is released.
                const unsigned long long t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 200000ull) sleep_ns(10000);
            }
        } else if (warp == 1 && rank == 0) {
            // --------------------------------------------------- MMA issuer --
            // The whole warp walks the loop and one elected lane issues, so that
            // addresses and descriptors stay in uniform registers: the issuing
            // thread's own time per 64 k has to stay below the MMAs' (384 clocks
            // at 192 columns).
            uint32_t slot = 0, slot_phase = 0;
            uint32_t local = 0;  // accumulators filled
            bool ok = true, issued = false, is_ready = false;
            for (long long tile = cluster; ok && tile < tiles; tile += nclusters) {
                const GroupedTile t = row_tile(table, tile, args.tiles_f, args.K);
                const uint32_t idesc = mma_idesc(TcTraits<kDtF16>::kFmt, TcTraits<kDtF16>::kFmt, 256, t.bn);
                for (int h = 0; ok && h < 2 * num_kb; h += Cfg::CHUNK_HALVES) {
                    const uint32_t acc = local & 1, acc_phase = (local >> 1) & 1;
                    ++local;
                    ok = pair_wait<CL>(&tempty[acc], acc_phase ^ 1u, abort_flag, args.status, abort_local, rank);
                    if (!__all_sync(0xffffffffu, ok)) ok = false;
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + acc * acc_stride;
                    const int end = min(2 * num_kb, h + Cfg::CHUNK_HALVES);
                    for (int i = h; i < end; i += 2) {
                        if (!is_ready) {
                            ok = pair_wait<CL>(&ready[slot >> 1], slot_phase, abort_flag, args.status, abort_local,
                                               rank);
                            if (!__all_sync(0xffffffffu, ok)) ok = false;
                            if (!ok) break;
                        }
                        smem_acquire_cluster();
                        tc_fence_after();
                        // ask for the next two slots now: the answer comes while these MMAs issue
                        const uint32_t next = slot + 2 == slots ? 0u : slot + 2;
                        const uint32_t next_phase = next == 0 ? slot_phase ^ 1u : slot_phase;
                        const bool next_ready = mbar_test_wait(smem_u32(&ready[next >> 1]), next_phase);
                        const uint64_t bd = sw128_desc(smem_u32(slot_base) + slot * sh.slot_bytes, 16u, 1024u);
                        const uint64_t bd2 = bd + (sh.slot_bytes >> 4);
                        const uint32_t w_tmem = w_slot0 + slot * Cfg::W_SLOT_COLS;
                        if (elect_one()) {
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)  // 16 k: 8 columns of W, 32 bytes of X's rows
                                tc_mma_pair_f16_tmem_a(d_tmem, w_tmem + ks * 8, bd + 2 * ks, idesc,
                                                       (i != h || ks != 0) ? 1u : 0u);
                            tc_commit_pair(&freed[slot], 0x3);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                tc_mma_pair_f16_tmem_a(d_tmem, w_tmem + Cfg::W_SLOT_COLS + ks * 8, bd2 + 2 * ks,
                                                       idesc, 1u);
                            tc_commit_pair(&freed[slot + 1], 0x3);
                            if (i + 2 == end) tc_commit_pair(&tfull[acc], 0x3);
                        }
                        issued = true;
                        is_ready = __all_sync(0xffffffffu, next_ready);
                        slot = next;
                        slot_phase = next_phase;
                    }
                }
            }
            if (*abort_flag && issued) {
                if (elect_one()) tc_commit_pair(mma_done, 1u);
                mbar_drain_wait(mma_done, 0, 100000000ull);
            }
        }
    } else if (warp < Cfg::EPI_WARP0) {
        // ----------------------------------------------------- converters --
        regs_decrease<Cfg::CONV_REGS>();
        const int quad = warp & 3, set = (warp - Cfg::CONV_WARP0) >> 2, hk = set & 1;
        constexpr int step = Cfg::SETS / 2;  // stages from one turn to the next
        // 16-byte unit u of a row sits at u ^ (row % 8).  This thread reads units
        // 4 hk .. 4 hk + 3 of row 32 quad + lane of W; of rows lane, lane + 32, ... of
        // X it reads unit 4 hk + quad and writes units 2 quad and 2 quad + 1.
        const uint32_t sw = lane & 7;
        const uint32_t w_at = smem_u32(smem) + (quad * 32 + lane) * 128 + ((4 * hk ^ sw) << 4);
        const uint32_t x_at = smem_u32(smem) + Cfg::W_BYTES + lane * 128 + (((4 * hk + quad) ^ sw) << 4);
        const uint32_t xs_at = smem_u32(slot_base) + lane * 128 + ((2 * quad ^ sw) << 4);
        const uint32_t w_tmem0 = w_slot0 + (static_cast<uint32_t>(quad * 32) << 16);
        int kb = set >> 1;  // stage of the tile, numbered on through all tiles
        uint32_t stage = kb, phase = 0, slot = 2 * kb + hk, slot_phase = 0;
        bool ok = true;
        for (long long tile = cluster; ok && tile < tiles; tile += nclusters, kb -= num_kb) {
            const int bnh = row_tile(table, tile, args.tiles_f, args.K).bn >> 1;
            for (; kb < num_kb; kb += step) {
                bool got = pair_wait<CL>(&full[stage], phase, abort_flag, args.status, abort_local, rank);
                const uint32_t st = stage * sh.stage_bytes;
                uint4 c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) c[i] = lds128((w_at + st) ^ (i << 4));
                got = got &&
                      pair_wait<CL>(&freed[slot], slot_phase ^ 1u, abort_flag, args.status, abort_local, rank);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // this row's 64 codes to 32 columns of tensor memory
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    uint32_t out[16];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        expand4(c[2 * p + i].x, out[8 * i], out[8 * i + 1]);
                        expand4(c[2 * p + i].y, out[8 * i + 2], out[8 * i + 3]);
                        expand4(c[2 * p + i].z, out[8 * i + 4], out[8 * i + 5]);
                        expand4(c[2 * p + i].w, out[8 * i + 6], out[8 * i + 7]);
                    }
                    tmem_st_x16(w_tmem0 + slot * Cfg::W_SLOT_COLS + p * 16, out);
                }
                // 16 codes of each row of X; rows of a started 32 past the tile's hold what
                // the stage held before, and no MMA reads what becomes of them
                const uint32_t xs = xs_at + slot * sh.slot_bytes;
                constexpr int XR = kI8TileRows / 64;  // most rows per thread
#pragma unroll
                for (int i = 0; i < XR; ++i)
                    if (32 * i < bnh) c[i] = lds128(x_at + st + i * 32 * 128);
#pragma unroll
                for (int i = 0; i < XR; ++i) {
                    if (32 * i < bnh) {
                        uint4 a, b;
                        expand4(c[i].x, a.x, a.y);
                        expand4(c[i].y, a.z, a.w);
                        expand4(c[i].z, b.x, b.y);
                        expand4(c[i].w, b.z, b.w);
                        sts128(xs + i * 32 * 128, a);
                        sts128((xs ^ 16) + i * 32 * 128, b);
                    }
                }
                tmem_st_wait();
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    smem_release_cluster();
                    mbar_arrive_remote_relaxed(ready0_leader + 8u * (slot >> 1));
                    mbar_arrive(&empty[stage]);
                }
                if ((slot += 2 * step) >= slots) {
                    slot -= slots;
                    slot_phase ^= 1u;
                }
                if ((stage += step) >= stages) {
                    stage -= stages;
                    phase ^= 1u;
                }
            }
        }
    } else {
        // ------------------------------------------------------- epilogue --
        regs_increase<Cfg::EPI_REGS>();
        using OutT = typename Elem<OUT>::T;
        const int quad = warp & 3, side = (warp - Cfg::EPI_WARP0) >> 2;
        const StoreArgs e{args.ldc, args.alpha, args.beta, args.epi};
        constexpr int MC = kI8TileRows / 64;  // most 32-column chunks of a warp
        uint32_t local = 0;
        bool ok = true;
        for (long long tile = cluster; ok && tile < tiles; tile += nclusters) {
            const GroupedTile t = row_tile(table, tile, args.tiles_f, args.K);
            const int chunks = t.bn >> 5;
            const int c_begin = side ? (chunks + 1) >> 1 : 0, nch = (side ? chunks : (chunks + 1) >> 1) - c_begin;
            const int f = t.f0 + static_cast<int>(rank) * 128 + quad * 32 + lane;
            const long long gf = static_cast<long long>(t.g) * args.F + f;
            const bool f_ok = f < args.F;
            const float bias = args.epi != kEpiNone && f_ok ? args.bias[gf] : 0.0f;
            const float cs = args.col_scale != nullptr && f_ok ? args.col_scale[gf] : 1.0f;
            OutT *out = static_cast<OutT *>(args.C) + t.r0 * args.ldc + f;
            const uint32_t t_quad = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + c_begin * 32;
            auto store = [&](float (&v)[32], int c) {
                const int row = (c_begin + c) * 32;
                OutT *c0 = out + row * args.ldc;
                chunk_values_t<OUT>(v, c0, args.F - f, t.nr - row,
                                    args.row_scale != nullptr ? args.row_scale + t.r0 + row : nullptr, cs, bias, e);
                store_chunk_t<OUT>(v, c0, args.F - f, t.nr - row, args.ldc);
            };
            auto accumulator = [&](uint32_t &acc) {  // the next one; false when the kernel gives up
                acc = local & 1;
                const uint32_t acc_phase = (local >> 1) & 1;
                ++local;
                ok = __all_sync(0xffffffffu,
                                pair_wait<CL>(&tfull[acc], acc_phase, abort_flag, args.status, abort_local, rank));
                if (ok) tc_fence_after();
                return ok;
            };
            auto release = [&](uint32_t acc) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(tempty0_leader + 8u * acc);
            };
            uint32_t acc;
            if (2 * num_kb <= Cfg::CHUNK_HALVES) {
                // one accumulator holds the whole sum, exact in fp32
                if (!accumulator(acc)) break;
#pragma unroll 1
                for (int c = 0; c < nch; ++c) {
                    uint32_t raw[32];
                    __syncwarp();
                    tmem_ld_issue(t_quad + acc * acc_stride + c * 32, raw);
                    tmem_ld_wait(raw);
                    if (c + 1 == nch) release(acc);
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]);
                    store(v, c);
                }
                if (nch == 0) release(acc);
                continue;
            }
            int sum[MC][32];
#pragma unroll
            for (int c = 0; c < MC; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[c][j] = 0;
            for (int h = 0; h < 2 * num_kb; h += Cfg::CHUNK_HALVES) {
                if (!accumulator(acc)) break;
#pragma unroll
                for (int c = 0; c < MC; ++c) {
                    if (c < nch) {
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            uint32_t raw[16];
                            __syncwarp();
                            tmem_ld_x16(t_quad + acc * acc_stride + c * 32 + p * 16, raw);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                sum[c][16 * p + j] += __float2int_rn(__uint_as_float(raw[j]));
                        }
                    }
                }
                release(acc);
            }
            if (!ok) break;
#pragma unroll
            for (int c = 0; c < MC; ++c) {
                if (c < nch) {
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __int2float_rn(sum[c][j]);
                    store(v, c);
                }
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    cluster_sync_all();  // no CTA leaves while its peer may still signal into it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
    }
}

template <int OUT>
cudaError_t launch_i8_tc_out(const CUtensorMap &tw, const CUtensorMap &tx32, const CUtensorMap &tx16,
                             const GtcArgs &a, int clusters, cudaStream_t stream) {
    auto kern = i8_tc_kernel<OUT>;
    cudaError_t err =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, I8Config::SMEM_MAX);
    if (err != cudaSuccess) return err;
    // The register trade adds up for this launch count only.  The build holds the compiler to it; a library
    // built past that check refuses here, where the kernel would wait for registers for ever.
    cudaFuncAttributes fa;
    if ((err = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return err;
    if (fa.numRegs != I8Config::LAUNCH_REGS) return cudaErrorInvalidKernelImage;
    GtcArgs args = a;
    if (args.most < 64 || args.most > kI8TileRows || args.most % 64 != 0) return cudaErrorInvalidValue;
    args.stages = I8Config::MAX_STAGES;
    while (args.stages > 4 && I8Config::fixed_bytes(args.G) + I8Shape(args.most, args.stages).bytes() > I8Config::SMEM_MAX)
        --args.stages;
    const int smem = I8Config::fixed_bytes(args.G) + I8Shape(args.most, args.stages).bytes();
    if (smem > I8Config::SMEM_MAX || smem <= I8Config::SMEM_MAX / 2) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters, 1, 1);
    cfg.blockDim = dim3(I8Config::THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, tw, tx32, tx16, args);
}

}  // namespace

cudaError_t launch_i8_tc(int out, const CUtensorMap &tw, const CUtensorMap &tx32, const CUtensorMap &tx16,
                         const GtcArgs &args, int clusters, cudaStream_t stream) {
    if (out == kDtF32) return launch_i8_tc_out<kDtF32>(tw, tx32, tx16, args, clusters, stream);
    if (out == kDtF16) return launch_i8_tc_out<kDtF16>(tw, tx32, tx16, args, clusters, stream);
    if (out == kDtBF16) return launch_i8_tc_out<kDtBF16>(tw, tx32, tx16, args, clusters, stream);
    return cudaErrorInvalidValue;
}

}  // namespace gb300
