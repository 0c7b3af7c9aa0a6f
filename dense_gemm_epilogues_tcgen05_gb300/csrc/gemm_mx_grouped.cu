// gemm_mx_grouped.cu -- the block-scaled ("MX") product grouped by expert, on
// pairs of SMs (tcgen05 cta_group::2).
//
//   C[r][f] = act(alpha rs[r] sum_k x[r][k] w[g][f][k] + beta C[r][f] + bias[g][f])
//
// over the rows r of group g, x and w E4M3 or E2M1 elements with an E8M0 scale per
// 32 k, applied by the tensor cores from tensor memory.  Computed transposed as in
// gemm_grouped_tc.cu: the MMA's 256 rows are the weights' output channels, its
// columns up to kMost rows of a group in steps of 32.
//
// Scales stay row-major in memory, as the quantiser writes them; a group may begin
// at any row, so that no layout made beforehand would fit its tiles.  A box of 16
// scales (512 k) of each row arrives by TMA in a ring of its own, and a warp
// turns it in place into the chunks that tcgen05.cp spreads over tensor memory:
// row 32 g + l, block 4 c + j of a 128-row block at byte 512 c + 16 l + 4 g + j
// (the four words that a lane reads of its rows, exchanged for the four it
// writes: no lane needs another's).
//
// Roles, per CTA:
//   warp 0       TMA producer: its 128 rows of W, its half of the tile's rows of X
//                (128 bytes of k a stage) counted on the leader's barrier; the
//                scales of its W rows and of all the tile's rows of X on its own;
//   warp 1       MMA issuer (leader CTA only), two accumulators;
//   warp 2       scales: lays a box out and tells the leader;
//   warps 3-10   epilogue: two per 32-lane quadrant of tensor memory, each half of
//                the tile's columns (store_chunk_t).
#include "gemm_tcgen05.cuh"
#include "grouped.cuh"
#include "mx_traits.cuh"

namespace gb300 {

namespace {

template <int ELEM>
struct MxgConfig {
    static constexpr int STAGES = 6, ENTRIES = 4;               // operand ring, scale ring
    static constexpr int CHUNKS = MxTraits<ELEM>::kChunks;      // 128-k scale chunks of a stage
    static constexpr int KPE = 4 / CHUNKS;                      // stages of a scale box (512 k)
    static constexpr int A_BYTES = 128 * 128, B_BYTES = kMxgMost / 2 * 128, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int SFA_BYTES = 128 * 16, ENTRY_BYTES = SFA_BYTES + 256 * 16;
    static constexpr int ACC_STRIDE = kMxgMost, TMEM_COLS = 512;
    static constexpr int SF_COLS = 12 * CHUNKS, SF_SLOTS = 2;   // W: 4 per chunk, X: 8 per chunk
    static constexpr int EPI_WARP0 = 3, EPI_WARPS = 8;
    static constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
    static constexpr int BAR_BYTES = 256, SMEM_MAX = 232448;
    static_assert(2 * ACC_STRIDE + SF_SLOTS * SF_COLS <= TMEM_COLS, "accumulators and scale slots fit");
    static_assert((2 * STAGES + 3 * ENTRIES + 5) * 8 + 8 <= BAR_BYTES, "barriers fit their slot");
    static_assert(B_BYTES % 1024 == 0 && STAGE_BYTES % 1024 == 0, "swizzle atoms stay aligned");
    // after up to 1023 bytes of alignment: [stages][scale boxes][barriers][group table]
    static int smem_bytes(int G) {
        return 1024 + STAGES * STAGE_BYTES + ENTRIES * ENTRY_BYTES + BAR_BYTES + (group_table_bytes(G) + 15) / 16 * 16;
    }
    static_assert(1024 + STAGES * STAGE_BYTES + ENTRIES * ENTRY_BYTES + BAR_BYTES + group_table_bytes(kMaxGroups) + 16 <=
                      SMEM_MAX, "fits the 227 KB opt-in shared memory");
};

// A 128-row block of scales, row-major in rows of 16 bytes, to four chunks in its place.  Warp-collective.
__device__ __forceinline__ void lay_out_scales(uint32_t addr) {
    const uint32_t lane16 = (threadIdx.x & 31) * 16;
    const uint4 r0 = lds128(addr + lane16), r1 = lds128(addr + 512 + lane16), r2 = lds128(addr + 1024 + lane16),
                r3 = lds128(addr + 1536 + lane16);
    sts128(addr + lane16, make_uint4(r0.x, r1.x, r2.x, r3.x));
    sts128(addr + 512 + lane16, make_uint4(r0.y, r1.y, r2.y, r3.y));
    sts128(addr + 1024 + lane16, make_uint4(r0.z, r1.z, r2.z, r3.z));
    sts128(addr + 1536 + lane16, make_uint4(r0.w, r1.w, r2.w, r3.w));
}

template <int ELEM, int OUT>
__global__ void __launch_bounds__(MxgConfig<ELEM>::THREADS, 1)
    mx_grouped_kernel(const __grid_constant__ MxgMaps maps, const __grid_constant__ GtcArgs args) {
    using Cfg = MxgConfig<ELEM>;
    constexpr int CL = 2;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char *entries = smem + Cfg::STAGES * Cfg::STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(entries + Cfg::ENTRIES * Cfg::ENTRY_BYTES);
    uint64_t *empty = full + Cfg::STAGES;
    uint64_t *landed = empty + Cfg::STAGES;       // this CTA's scale box has landed
    uint64_t *ready = landed + Cfg::ENTRIES;      // (leader's) both CTAs' boxes are laid out
    uint64_t *sempty = ready + Cfg::ENTRIES;      // the MMAs of the box are done
    uint64_t *tfull = sempty + Cfg::ENTRIES;
    uint64_t *tempty = tfull + 2;
    uint64_t *mma_done = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();  // 0: leader
    const int cluster = blockIdx.x / CL, nclusters = gridDim.x / CL;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < Cfg::ENTRIES; ++s) {
            mbar_init(&landed[s], 1);
            mbar_init(&ready[s], CL);
            mbar_init(&sempty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], CL * Cfg::EPI_WARPS);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&maps.w);
        tma_prefetch_desc(&maps.ws);
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
        threadIdx.x, Cfg::THREADS, RowTilesOf{args.most});
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t full0_leader = mapa_shared(smem_u32(&full[0]), 0);
    const uint32_t ready0_leader = mapa_shared(smem_u32(&ready[0]), 0);
    const uint32_t tempty0_leader = mapa_shared(smem_u32(&tempty[0]), 0);
    const uint32_t abort_local = smem_u32(const_cast<int *>(abort_flag));
    const int num_kb = (args.K / (ELEM == kMxE2M1 ? 2 : 1) + 127) / 128;
    const long long tiles = static_cast<long long>(table.first[args.G]) * args.tiles_f;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer --
            uint32_t stage = 0, phase = 0, entry = 0, ephase = 0;
            bool ok = true, issued = false;
            const uint64_t keep = l2_policy_evict_last();
            for (long long tile = cluster; ok && tile < tiles; tile += nclusters) {
                const GroupedTile t = row_tile(table, tile, args.tiles_f, args.K);
                const int f = t.f0 + static_cast<int>(rank) * 128;
                const int bnh = t.bn >> 1;
                const int c0 = t.r0 + static_cast<int>(rank) * bnh;  // first of this CTA's MMA columns
                const uint32_t bytes = Cfg::A_BYTES + bnh * 128u;
                const int sm = t.bn <= 32 ? 0 : t.bn <= 64 ? 1 : t.bn <= 128 ? 2 : 3;  // box of 32 << sm rows' scales
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (kb % Cfg::KPE == 0) {
                        if (!pair_wait<CL>(&sempty[entry], ephase ^ 1u, abort_flag, args.status, abort_local, rank)) {
                            ok = false;
                            break;
                        }
                        issued = true;
                        unsigned char *sf = entries + entry * Cfg::ENTRY_BYTES;
                        mbar_arrive_expect_tx(&landed[entry], Cfg::SFA_BYTES + (512u << sm));
                        const int b = kb / Cfg::KPE * 16;
                        tma_load_3d_hint(sf, &maps.ws, &landed[entry], b, f, t.g, keep);
                        tma_load_2d_hint(sf + Cfg::SFA_BYTES, &maps.xs[sm], &landed[entry], b, t.r0, keep);
                        if (++entry == Cfg::ENTRIES) {
                            entry = 0;
                            ephase ^= 1u;
                        }
                    }
                    if (!pair_wait<CL>(&empty[stage], phase ^ 1u, abort_flag, args.status, abort_local, rank)) {
                        ok = false;
                        break;
                    }
                    issued = true;
                    unsigned char *sA = smem + stage * Cfg::STAGE_BYTES;
                    const uint32_t fbar = full0_leader + 8u * stage;
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2u * bytes);
                    tma_load_3d_pair(sA, &maps.w, fbar, kb * 128, f, t.g, keep);
                    tma_load_3d_pair(sA + Cfg::A_BYTES, &maps.x[(bnh >> 4) - 1], fbar, kb * 128, c0, 0, keep);
                    if (++stage == Cfg::STAGES) {
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
            // addresses and descriptors stay in uniform registers.
            const uint64_t a_desc0 = sw128_desc(smem_u32(smem), 16u, 1024u);
            const uint64_t b_desc0 = sw128_desc(smem_u32(smem) + Cfg::A_BYTES, 16u, 1024u);
            const uint64_t sf_desc0 = plain16_desc(smem_u32(entries));
            uint32_t stage = 0, phase = 0, entry = 0, ephase = 0, slot = 0;
            bool ok = true, issued = false;
            int local = 0;
            for (long long tile = cluster; ok && tile < tiles; tile += nclusters) {
                if (num_kb == 0) break;  // the epilogue alone
                const GroupedTile t = row_tile(table, tile, args.tiles_f, args.K);
                const uint32_t acc = local & 1, acc_phase = (local >> 1) & 1;
                ++local;
                ok = pair_wait<CL>(&tempty[acc], acc_phase ^ 1u, abort_flag, args.status, abort_local, rank);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * Cfg::ACC_STRIDE;
                for (int kb = 0; kb < num_kb; ++kb) {
                    const int part = kb % Cfg::KPE;  // of the scale box
                    if (part == 0) {
                        ok = pair_wait<CL>(&ready[entry], ephase, abort_flag, args.status, abort_local, rank);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        smem_acquire_cluster();
                    }
                    ok = pair_wait<CL>(&full[stage], phase, abort_flag, args.status, abort_local, rank);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = stage * (Cfg::STAGE_BYTES >> 4);  // addresses are in 16-byte units, below 2^14
                    const uint64_t ad = a_desc0 + at, bd = b_desc0 + at;
                    const uint64_t sd = sf_desc0 + entry * (Cfg::ENTRY_BYTES >> 4);
                    const uint32_t sfa = tmem_base + 2 * Cfg::ACC_STRIDE + slot * Cfg::SF_COLS, sfb = sfa + 4 * Cfg::CHUNKS;
                    const bool last = kb + 1 == num_kb, box_done = last || part + 1 == Cfg::KPE;
                    if (elect_one()) {
#pragma unroll
                        for (int c = 0; c < Cfg::CHUNKS; ++c) {
                            const uint64_t ch = sd + static_cast<uint32_t>(part * Cfg::CHUNKS + c) * 32u;
                            tc_cp_32x128b_x4_pair(sfa + 4 * c, ch);
                            tc_cp_32x128b_x4_pair(sfb + 8 * c, ch + (Cfg::SFA_BYTES >> 4));
                            if (t.bn > 128) tc_cp_32x128b_x4_pair(sfb + 8 * c + 4, ch + ((Cfg::SFA_BYTES + 2048) >> 4));
                        }
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            const uint32_t chunk = Cfg::CHUNKS == 1 ? 0u : static_cast<uint32_t>(ks >> 1);
                            const uint32_t sf_id = Cfg::CHUNKS == 1 ? static_cast<uint32_t>(ks)
                                                                    : static_cast<uint32_t>((ks & 1) * 2);
                            const uint32_t idesc = mma_idesc_bs(MxTraits<ELEM>::kFmt, 256, t.bn, sf_id, sf_id);
                            tc_mma_bs_pair<MxTraits<ELEM>::kKind>(d_tmem, ad + ks * 2, bd + ks * 2, idesc, sfa + 4 * chunk,
                                                                   sfb + 8 * chunk, (kb | ks) != 0 ? 1u : 0u);
                        }
                        tc_commit_pair(&empty[stage], 0x3);
                        if (box_done) tc_commit_pair(&sempty[entry], 0x3);
                        if (last) tc_commit_pair(&tfull[acc], 0x3);
                    }
                    __syncwarp();
                    issued = true;
                    slot ^= 1u;
                    if (box_done && ++entry == Cfg::ENTRIES) {
                        entry = 0;
                        ephase ^= 1u;
                    }
                    if (++stage == Cfg::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (*abort_flag && issued) {
                if (elect_one()) tc_commit_pair(mma_done, 1u);
                mbar_drain_wait(mma_done, 0, 100000000ull);
            }
        }
    } else if (warp == 2) {
        // -------------------------------------------------------- scales --
        uint32_t entry = 0, ephase = 0;
        bool ok = true;
        for (long long tile = cluster; ok && tile < tiles; tile += nclusters) {
            const GroupedTile t = row_tile(table, tile, args.tiles_f, args.K);
            for (int kb = 0; kb < num_kb; kb += Cfg::KPE) {
                const bool got = pair_wait<CL>(&landed[entry], ephase, abort_flag, args.status, abort_local, rank);
                ok = __all_sync(0xffffffffu, got);
                if (!ok) break;
                const uint32_t sf = smem_u32(entries + entry * Cfg::ENTRY_BYTES);
                lay_out_scales(sf);
                // (rows past the box are an earlier tile's scales or none: their columns are not stored)
                lay_out_scales(sf + Cfg::SFA_BYTES);
                if (t.bn > 128) lay_out_scales(sf + Cfg::SFA_BYTES + 2048);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    smem_release_cluster();
                    mbar_arrive_remote_relaxed(ready0_leader + 8u * entry);
                }
                if (++entry == Cfg::ENTRIES) {
                    entry = 0;
                    ephase ^= 1u;
                }
            }
        }
    } else {
        // ------------------------------------------------------- epilogue --
        using OutT = typename Elem<OUT>::T;
        const int quad = warp & 3;                      // TMEM lanes 32*quad ..
        const int half = (warp - Cfg::EPI_WARP0) >> 2;  // which half of the tile's columns
        const StoreArgs e{args.ldc, args.alpha, args.beta, args.epi};
        int local = 0;
        for (long long tile = cluster; tile < tiles; tile += nclusters) {
            const GroupedTile t = row_tile(table, tile, args.tiles_f, args.K);
            const int f = t.f0 + static_cast<int>(rank) * 128 + quad * 32 + lane;
            const float bias = (e.epi != kEpiNone && f < args.F)
                                   ? args.bias[static_cast<long long>(t.g) * args.F + f] : 0.0f;
            OutT *c = static_cast<OutT *>(args.C) + t.r0 * args.ldc + f;
            const float *rs = args.row_scale != nullptr ? args.row_scale + t.r0 : nullptr;
            const int chunks = t.bn >> 5;
            const int c_begin = half ? (chunks + 1) >> 1 : 0, nch = (half ? chunks : (chunks + 1) >> 1) - c_begin;
            const uint32_t t_quad = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + c_begin * 32;
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
                const int row = (c_begin + ch) * 32;
                OutT *c0 = c + row * args.ldc;
                chunk_values_t<OUT>(v, c0, args.F - f, t.nr - row, rs != nullptr ? rs + row : nullptr, 1.0f, bias, e);
                store_chunk_t<OUT>(v, c0, args.F - f, t.nr - row, args.ldc);
            }
            if (num_kb > 0 && nch == 0) {  // a 32-column tile has no second half
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(tempty0_leader + 8u * acc);
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

template <int ELEM, int OUT>
cudaError_t launch_mxg(const MxgMaps &maps, const GtcArgs &args, int clusters, cudaStream_t stream) {
    using Cfg = MxgConfig<ELEM>;
    auto kern = mx_grouped_kernel<ELEM, OUT>;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_MAX);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters, 1, 1);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::smem_bytes(args.G);
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

template <int ELEM>
cudaError_t launch_mxg_out(int out, const MxgMaps &maps, const GtcArgs &args, int clusters, cudaStream_t stream) {
    if (out == kDtF32) return launch_mxg<ELEM, kDtF32>(maps, args, clusters, stream);
    if (out == kDtF16) return launch_mxg<ELEM, kDtF16>(maps, args, clusters, stream);
    if (out == kDtBF16) return launch_mxg<ELEM, kDtBF16>(maps, args, clusters, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_mx_grouped(int elem, int out, const MxgMaps &maps, const GtcArgs &args, int clusters,
                              cudaStream_t stream) {
    if (elem == kMxE4M3) return launch_mxg_out<kMxE4M3>(out, maps, args, clusters, stream);
    if (elem == kMxE2M1) return launch_mxg_out<kMxE2M1>(out, maps, args, clusters, stream);
    return cudaErrorInvalidValue;
}

}  // namespace gb300
