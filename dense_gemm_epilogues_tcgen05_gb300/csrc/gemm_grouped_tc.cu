// gemm_grouped_tc.cu -- products grouped by expert on pairs of SMs (tcgen05
// cta_group::2), forward and weight gradient.
//
//   forward    C[r][f] = sum_k A[r][k] B[g][k][f] over the rows r of group g
//   gradient   C[g][m][f] = sum_r A[r][m] D[r][f] over the rows r of group g
//
// Both are computed transposed: the MMA's 256 rows are columns f of C (the
// weights' output channels; the gradient's contiguous index) and its up to 256
// columns are the rows of C (tokens; the index m).  The ragged index is then
// the MMA's N, whose width a tile chooses at run time in steps of 32: a group
// of m rows takes ceil(m / 256) tiles of one common width, so 300 rows cost
// two tiles of 160 columns, and 5 rows one of 32, where 256-row tiles of
// tokens would compute 512 and 256.  In the gradient the ragged index is the
// summed one.
//
// One persistent cluster of two CTAs per SM pair walks the tiles, which it
// finds from `offsets` itself (grouped.cuh).  Roles, per CTA:
//
//   warp 0       TMA producer: its own 128 rows of the MMA's first operand and
//                its own half of the columns' operand, 64 deep, into a ring of
//                seven (six beside a large group table) 32 KB stages, counted on
//                the leader's barrier;
//   warp 1       MMA issuer (leader CTA only), two 256-column accumulators;
//   warp 2       gradient only: the last k-block of a group reaches into the
//                next group's rows (or past T).  They are zeroed in shared
//                memory before the MMA reads them -- in both operands, since
//                zero times a neighbour's infinity or NaN would be NaN.  Such
//                a block is loaded on a barrier of its own CTA, warp 2 clears
//                rows valid .. 63 and arrives on the leader's `fixed` barrier;
//   warps 3-10   epilogue: two per 32-lane quadrant of tensor memory, each
//                half of the tile's columns (store_chunk_t).
//
// Bound and measured (GB300): small groups by the weights' bytes, each expert's
// read once per 256 of its rows and from L2 after the first (64 experts x 4096 rows,
// 2048 x 4096 fp16: 173 us, 6.5 TB/s of the 1.12 GB); large ones by the tensor pipe
// (32 experts, 32768 rows, 4096 x 4096 bf16, row gradient: 748 us,
// 1.47 PFLOP/s; 3 % faster without the fp32 sums in registers); the gradient by the tensor pipe and its output's
// bytes together (16 experts, 16384 rows, 2048 x 4096, fp32 out: 201 us, 61 % tensor pipe,
// 738 MB), and by its tiles' fixed costs when groups are small (24 gradients of
// 1000 x 1000 over 777 rows: 25 us with the bias sums).
#include "gemm_tcgen05.cuh"
#include "grouped.cuh"

namespace gb300 {

namespace {

struct GtcConfig {
    static constexpr int BK = 64, MAX_STAGES = 7;
    static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int EPI_WARP0 = 3, EPI_WARPS = 8;
    static constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
    static constexpr int TMEM_COLS = 512, ACC_STRIDE = 256;
    static constexpr int BAR_BYTES = 320, SMEM_MAX = 232448;
    // k-blocks summed in the tensor core's accumulator before the sum moves to registers
    static constexpr int SEG = 8;
    static_assert((4 * MAX_STAGES + 5) * 8 + 8 <= BAR_BYTES, "barriers fit their slot");
    // after up to 1023 bytes of alignment: [stages][barriers][group table]
    static int fixed_bytes(int G) { return 1024 + BAR_BYTES + (group_table_bytes(G) + 15) / 16 * 16; }
};
static_assert(1024 + GtcConfig::BAR_BYTES + group_table_bytes(kMaxGroups) + 6 * GtcConfig::STAGE_BYTES <=
                  GtcConfig::SMEM_MAX, "six stages always fit");

// Walks this cluster's tiles.
template <bool WG>
struct GtcIter {
    const GroupTable &t;
    const GtcArgs &a;
    long long tile, tiles;
    int step;
    __device__ __forceinline__ GtcIter(const GroupTable &t_, const GtcArgs &a_, int cluster, int nclusters)
        : t(t_), a(a_), tile(cluster), step(nclusters) {
        tiles = WG ? static_cast<long long>(a.G) * a.tiles_r * a.tiles_f
                   : static_cast<long long>(t.first[a.G]) * a.tiles_f;
    }
    __device__ __forceinline__ bool next(GroupedTile &o) {
        if (tile >= tiles) return false;
        if constexpr (WG) {
            const int rt = static_cast<int>(tile / a.tiles_f);
            o.f0 = static_cast<int>(tile - static_cast<long long>(rt) * a.tiles_f) * 256;
            o.g = rt / a.tiles_r;
            const int in = rt - o.g * a.tiles_r;
            const int w = tile_width(a.R, a.tiles_r);
            o.r0 = in * w;
            o.nr = min(w, a.R - o.r0);
            o.bn = (o.nr + 31) & ~31;
            o.k0 = t.lo[o.g];
            o.nk = t.hi[o.g] - o.k0;
        } else {
            o = row_tile(t, tile, a.tiles_f, a.K);
        }
        tile += step;
        return true;
    }
};

template <bool WG, int AB, int OUT>
__global__ void __launch_bounds__(GtcConfig::THREADS, 1)
    grouped_tc_kernel(const __grid_constant__ GtcMaps maps, const __grid_constant__ GtcArgs args) {
    using Cfg = GtcConfig;
    constexpr int BK = Cfg::BK, CL = 2;
    const uint32_t stages = args.stages;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + stages * Cfg::STAGE_BYTES);
    uint64_t *empty = full + Cfg::MAX_STAGES;
    uint64_t *landed = empty + Cfg::MAX_STAGES;   // gradient, last k-blocks: this CTA's bytes have landed
    uint64_t *fixed = landed + Cfg::MAX_STAGES;   // (leader's) both CTAs have cleared the foreign rows
    uint64_t *tfull = fixed + Cfg::MAX_STAGES;
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
            mbar_init(&empty[s], 1);
            mbar_init(&landed[s], 1);
            mbar_init(&fixed[s], CL);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], CL * Cfg::EPI_WARPS);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&maps.a);
        tma_prefetch_desc(&maps.b[WG ? 2 : 7]);
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
    const GroupTable table = group_table_build(
        reinterpret_cast<int *>(reinterpret_cast<unsigned char *>(full) + Cfg::BAR_BYTES), args.offsets, args.G, args.T,
        threadIdx.x, Cfg::THREADS, RowTilesOf{256});
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t full0_leader = mapa_shared(smem_u32(&full[0]), 0);
    const uint32_t fixed0_leader = mapa_shared(smem_u32(&fixed[0]), 0);
    const uint32_t tempty0_leader = mapa_shared(smem_u32(&tempty[0]), 0);
    const uint32_t abort_local = smem_u32(const_cast<int *>(abort_flag));
    GtcIter<WG> it(table, args, cluster, nclusters);
    GroupedTile t;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer --
            uint32_t stage = 0, phase = 0;
            bool ok = true, issued = false;
            const uint64_t keep = l2_policy_evict_last();
            while (ok && it.next(t)) {
                const int f = t.f0 + static_cast<int>(rank) * 128;
                const int bnh = t.bn >> 1;
                const int c0 = t.r0 + static_cast<int>(rank) * bnh;  // first of this CTA's MMA columns
                const int num_kb = (t.nk + BK - 1) / BK;
                const bool b_whole = WG && args.b_whole && (c0 & 63) == 0;
                const uint32_t bytes = Cfg::A_BYTES + (WG ? ((bnh + 63) >> 6) * 64u * 128u : bnh * 128u);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!pair_wait<CL>(&empty[stage], phase ^ 1u, abort_flag, args.status, abort_local, rank)) {
                        ok = false;
                        break;
                    }
                    issued = true;
                    unsigned char *sA = smem + stage * Cfg::STAGE_BYTES;
                    unsigned char *sB = sA + Cfg::A_BYTES;
                    const int k = t.k0 + kb * BK;
                    // One load per operand wherever a map allows: each takes the issuing
                    // thread about 90 clocks, and a k-block's MMAs only 512.
                    if (WG && (kb + 1) * BK > t.nk) {
                        // reaches past the group: on this CTA's own barrier, for warp 2
                        if (rank == 0) mbar_arrive(&full[stage]);
                        mbar_arrive_expect_tx(&landed[stage], bytes);
                        if (args.a_whole)
                            tma_load_4d_hint(sA, &maps.a, &landed[stage], 0, k, f >> 6, 0, keep);
                        else
                            for (int j = 0; j < 2; ++j)
                                tma_load_3d_hint(sA + j * 64 * 128, &maps.a, &landed[stage], f + j * 64, k, 0, keep);
                        if (b_whole)
                            tma_load_4d_hint(sB, &maps.b[bnh > 64], &landed[stage], 0, k, c0 >> 6, 0, keep);
                        else
                            for (int j = 0; j * 64 < bnh; ++j)
                                tma_load_3d_hint(sB + j * 64 * 128, &maps.b[2], &landed[stage], c0 + j * 64, k, 0,
                                                 keep);
                    } else {
                        const uint32_t fbar = full0_leader + 8u * stage;
                        if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2u * bytes);
                        if (!WG && !args.a_mn) {
                            tma_load_3d_pair(sA, &maps.a, fbar, k, f, t.g, keep);
                        } else if (args.a_whole) {
                            tma_load_4d_pair(sA, &maps.a, fbar, 0, k, f >> 6, WG ? 0 : t.g, keep);
                        } else {
                            for (int j = 0; j < 2; ++j)
                                tma_load_3d_pair(sA + j * 64 * 128, &maps.a, fbar, f + j * 64, k, WG ? 0 : t.g, keep);
                        }
                        if (!WG) {
                            tma_load_3d_pair(sB, &maps.b[(bnh >> 4) - 1], fbar, k, c0, 0, keep);
                        } else if (b_whole) {
                            tma_load_4d_pair(sB, &maps.b[bnh > 64], fbar, 0, k, c0 >> 6, 0, keep);
                        } else {
                            for (int j = 0; j * 64 < bnh; ++j)
                                tma_load_3d_pair(sB + j * 64 * 128, &maps.b[2], fbar, c0 + j * 64, k, 0, keep);
                        }
                    }
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
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ---------------------------------------------------- MMA issuer --
            // The whole warp walks the loop and one elected lane issues, so that
            // addresses and descriptors stay in uniform registers, and the next stage
            // is asked for before this one's MMAs issue: a k-block's MMAs take 512
            // clocks, and the issuing thread's own time has to stay well below.
            const uint32_t a_mn = WG ? 1u : args.a_mn, b_mn = WG ? 1u : 0u;
            const uint32_t a_kstep = (a_mn ? 128u * 16 : 32u) >> 4, b_kstep = (b_mn ? 128u * 16 : 32u) >> 4;
            const uint64_t a_desc0 = sw128_desc(smem_u32(smem), a_mn ? 128u * BK : 16u, 1024u);
            const uint64_t b_desc0 = sw128_desc(smem_u32(smem) + Cfg::A_BYTES, b_mn ? 128u * BK : 16u, 1024u);
            uint32_t stage = 0, phase = 0, fixed_parity = 0;
            bool ok = true, issued = false, is_full = false;
            int local = 0;
            while (ok && it.next(t)) {
                const int num_kb = (t.nk + BK - 1) / BK;
                if (num_kb == 0) continue;  // a group without rows: the epilogue alone
                const uint32_t idesc = mma_idesc(TcTraits<AB>::kFmt, TcTraits<AB>::kFmt, 256, t.bn) | (a_mn << 15) |
                                       (b_mn << 16);
                uint32_t acc = 0;
                for (int kb = 0; kb < num_kb; ++kb) {
                    const bool opens = kb % Cfg::SEG == 0;
                    if (opens) {
                        acc = local & 1;
                        const uint32_t acc_phase = (local >> 1) & 1;
                        ++local;
                        ok = pair_wait<CL>(&tempty[acc], acc_phase ^ 1u, abort_flag, args.status, abort_local, rank);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    if (!is_full) {
                        ok = pair_wait<CL>(&full[stage], phase, abort_flag, args.status, abort_local, rank);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                    }
                    if (WG && (kb + 1) * BK > t.nk) {
                        ok = pair_wait<CL>(&fixed[stage], (fixed_parity >> stage) & 1u, abort_flag, args.status,
                                           abort_local, rank);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        smem_acquire_cluster();
                        fixed_parity ^= 1u << stage;
                    }
                    tc_fence_after();
                    const uint32_t next = stage + 1 == stages ? 0u : stage + 1;
                    const uint32_t next_phase = next == 0 ? phase ^ 1u : phase;
                    const bool next_full = mbar_test_wait(smem_u32(&full[next]), next_phase);
                    const uint32_t d_tmem = tmem_base + acc * Cfg::ACC_STRIDE;
                    const uint32_t at = stage * (Cfg::STAGE_BYTES >> 4);  // addresses are in 16-byte units, below 2^14
                    const uint64_t ad = a_desc0 + at, bd = b_desc0 + at;
                    const bool closes = kb + 1 == num_kb || (kb + 1) % Cfg::SEG == 0;
                    if (elect_one()) {
#pragma unroll
                        for (uint32_t ks = 0; ks < BK / 16; ++ks)
                            tc_mma_pair<kKindF16>(d_tmem, ad + ks * a_kstep, bd + ks * b_kstep, idesc,
                                                  !opens || ks != 0 ? 1u : 0u);
                        tc_commit_pair(&empty[stage], 0x3);
                        if (closes) tc_commit_pair(&tfull[acc], 0x3);
                    }
                    issued = true;
                    is_full = __all_sync(0xffffffffu, next_full);
                    stage = next;
                    phase = next_phase;
                }
            }
            if (*abort_flag && issued) {
                if (elect_one()) tc_commit_pair(mma_done, 1u);
                mbar_drain_wait(mma_done, 0, 100000000ull);
            }
        }
    } else if (warp == 2) {
        if constexpr (WG) {
            // ------------------------------------------------ foreign rows --
            uint32_t stage = 0, parity = 0;
            bool ok = true;
            while (ok && it.next(t)) {
                const int num_kb = (t.nk + BK - 1) / BK;
                const int valid = t.nk - (num_kb - 1) * BK;  // rows of the last k-block
                if (num_kb > 0 && valid < BK) {
                    const uint32_t s = (stage + num_kb - 1) % stages;
                    const bool got =
                        pair_wait<CL>(&landed[s], (parity >> s) & 1u, abort_flag, args.status, abort_local, rank);
                    if (!__all_sync(0xffffffffu, got)) break;
                    parity ^= 1u << s;
                    // every operand box is 64 rows (k) of 128 bytes; a row's swizzle stays inside it
                    unsigned char *st = smem + s * Cfg::STAGE_BYTES;
                    const int boxes = 2 + (((t.bn >> 1) + 63) >> 6);
                    for (int b = 0; b < boxes; ++b) {
                        uint4 *row = reinterpret_cast<uint4 *>(st + b * 64 * 128 + valid * 128);
                        for (int i = lane; i < (BK - valid) * 8; i += 32) row[i] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        smem_release_cluster();
                        mbar_arrive_remote_relaxed(fixed0_leader + 8u * s);
                    }
                }
                stage = (stage + num_kb) % stages;
            }
        }
    } else {
        // ------------------------------------------------------- epilogue --
        using OutT = typename Elem<OUT>::T;
        const int quad = warp & 3;                      // TMEM lanes 32*quad ..
        const int half = (warp - Cfg::EPI_WARP0) >> 2;  // which half of the tile's columns
        // (a gradient has no activation: known here, their code stays out of its kernels)
        const StoreArgs e{args.ldc, args.alpha, args.beta, WG ? static_cast<int>(kEpiNone) : args.epi};
        int local = 0;
        while (it.next(t)) {
            const int num_kb = (t.nk + BK - 1) / BK;
            const int f = t.f0 + static_cast<int>(rank) * 128 + quad * 32 + lane;
            const float bias = (e.epi != kEpiNone && f < args.F)
                                   ? args.bias[static_cast<long long>(t.g) * args.F + f] : 0.0f;
            OutT *c = static_cast<OutT *>(args.C) + (WG ? t.g * args.scg : 0ll) + t.r0 * args.ldc + f;
            const float *rs = !WG && args.row_scale != nullptr ? args.row_scale + t.r0 : nullptr;
            const int chunks = t.bn >> 5;
            const int c_begin = half ? (chunks + 1) >> 1 : 0, nch = (half ? chunks : (chunks + 1) >> 1) - c_begin;
            const uint32_t t_quad = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + c_begin * 32;
            auto store = [&](float (&v)[32], int ch) {
                const int row = (c_begin + ch) * 32;
                OutT *c0 = c + row * args.ldc;
                chunk_values_t<OUT>(v, c0, args.F - f, t.nr - row, rs != nullptr ? rs + row : nullptr, 1.0f, bias, e);
                store_chunk_t<OUT>(v, c0, args.F - f, t.nr - row, args.ldc);
            };
            if (num_kb > Cfg::SEG) {
                // The tensor core's fp32 sums lose about half a unit in the last place per
                // instruction, always towards zero; over a few hundred of them that is an
                // error several times an fp32 sum's own (2048 rows: 1.4e-6 of the result; in a
                // bf16 row gradient 4096 deep it made 0.23 % of the outputs miss the nearest
                // bf16, where plain fp32 sums miss 0.04 %).  So every 512 k the accumulator is
                // added into registers, rounded to nearest.
                float sum[4][32];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[ch][j] = 0.0f;
                bool ok = true;
                for (int kb = 0; kb < num_kb; kb += Cfg::SEG) {
                    const uint32_t acc = local & 1, acc_phase = (local >> 1) & 1;
                    ++local;
                    const bool got = pair_wait<CL>(&tfull[acc], acc_phase, abort_flag, args.status, abort_local, rank);
                    ok = __all_sync(0xffffffffu, got);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        if (ch < nch) {
#pragma unroll
                            for (int p = 0; p < 2; ++p) {
                                uint32_t raw[16];
                                __syncwarp();
                                tmem_ld_x16(t_quad + acc * Cfg::ACC_STRIDE + ch * 32 + p * 16, raw);
#pragma unroll
                                for (int j = 0; j < 16; ++j) sum[ch][16 * p + j] += __uint_as_float(raw[j]);
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(tempty0_leader + 8u * acc);
                }
                if (!ok) break;
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
                    if (ch < nch) store(sum[ch], ch);
            } else {
                const uint32_t acc = local & 1, acc_phase = (local >> 1) & 1;
                if (num_kb > 0) {
                    ++local;
                    const bool got = pair_wait<CL>(&tfull[acc], acc_phase, abort_flag, args.status, abort_local, rank);
                    if (!__all_sync(0xffffffffu, got)) break;
                    tc_fence_after();
                }
#pragma unroll 1
                for (int ch = 0; ch < nch; ++ch) {
                    float v[32];
                    if (num_kb > 0) {
                        uint32_t raw[32];
                        __syncwarp();
                        tmem_ld_issue(t_quad + acc * Cfg::ACC_STRIDE + ch * 32, raw);
                        tmem_ld_wait(raw);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                    }
                    if (num_kb > 0 && ch + 1 == nch) {
                        // the accumulator is in registers: free it before the stores
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(tempty0_leader + 8u * acc);
                    }
                    store(v, ch);
                }
                if (num_kb > 0 && nch == 0) {  // a 32-column tile has no second half
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(tempty0_leader + 8u * acc);
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

template <bool WG, int AB, int OUT>
cudaError_t launch_gtc(const GtcMaps &maps, const GtcArgs &a, int clusters, cudaStream_t stream) {
    auto kern = grouped_tc_kernel<WG, AB, OUT>;
    GtcArgs args = a;
    args.stages = GtcConfig::MAX_STAGES;
    if (GtcConfig::fixed_bytes(args.G) + args.stages * GtcConfig::STAGE_BYTES > GtcConfig::SMEM_MAX) --args.stages;
    const int smem = GtcConfig::fixed_bytes(args.G) + args.stages * GtcConfig::STAGE_BYTES;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GtcConfig::SMEM_MAX);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters, 1, 1);
    cfg.blockDim = dim3(GtcConfig::THREADS, 1, 1);
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
    return cudaLaunchKernelEx(&cfg, kern, maps, args);
}

template <bool WG, int AB>
cudaError_t launch_gtc_out(int out, const GtcMaps &maps, const GtcArgs &args, int clusters, cudaStream_t stream) {
    if (out == kDtF32) return launch_gtc<WG, AB, kDtF32>(maps, args, clusters, stream);
    if (out == kDtF16) return launch_gtc<WG, AB, kDtF16>(maps, args, clusters, stream);
    if (out == kDtBF16) return launch_gtc<WG, AB, kDtBF16>(maps, args, clusters, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_grouped_tc(bool wgrad, int ab, int out, const GtcMaps &maps, const GtcArgs &args, int clusters, cudaStream_t stream) {
    if (ab == kDtF16)
        return wgrad ? launch_gtc_out<true, kDtF16>(out, maps, args, clusters, stream)
                     : launch_gtc_out<false, kDtF16>(out, maps, args, clusters, stream);
    if (ab == kDtBF16)
        return wgrad ? launch_gtc_out<true, kDtBF16>(out, maps, args, clusters, stream)
                     : launch_gtc_out<false, kDtBF16>(out, maps, args, clusters, stream);
    return cudaErrorInvalidValue;
}

}  // namespace gb300
