// gemm_mx_grouped.cu -- the block-scaled ("MX") product grouped by expert, on
// pairs of SMs (tcgen05 cta_group::2).
//
//   C[r][f] = act(alpha rs[r] sum_k x[r][k] w[g][f][k] + beta C[r][f] + bias[g][f])
//
// over the rows r of group g, x and w E4M3 or E2M1 elements with an E8M0 scale per
// 32 k, applied by the tensor cores from tensor memory.  Computed transposed as in
// gemm_grouped_tc.cu: the MMA's 256 rows are the weights' output channels, its
// columns up to kMxgMost rows of a group in steps of 16.
//
// Scales stay row-major in memory, as the quantiser writes them; a group may begin
// at any row, so that no layout made beforehand would fit its tiles.  A box of 16
// scales (512 k) of each row arrives by TMA, and a warp turns it in place into the
// chunks that tcgen05.cp spreads over tensor memory: row 32 g + l, block 4 c + j of
// a 128-row block at byte 512 c + 16 l + 4 g + j (the four words that a lane reads
// of its rows, exchanged for the four it writes: no lane needs another's).
//
// Roles, per CTA:
//   warp 0       loads (TMA) of its 128 rows of W, 128 bytes of k a stage, counted on
//                the leader's barrier;
//   warp 1       MMA issuer (leader CTA only), two accumulators;
//   warp 2       scales: lays out those of a pair of stages and arrives on the
//                leader's barrier;
//   warp 3       loads of its half of the tile's rows of X, and of the scales of its
//                rows of W and of all the tile's rows of X, on a barrier of its own;
//   warps 4-11   epilogue: two per 32-lane quadrant of tensor memory, each half of
//                the tile's columns (store_chunk_t).
//
// Sums: the tensor cores cut each instruction's sum off towards zero.  E4M3 products
// span 36 bits, so that nearly every instruction loses about half a unit in the last
// place: of the terms' absolute sum 3.9e-6 for 8192 of one sign, 2.0e-5 with elements
// four powers of ten apart (fp32 sums 4e-7 and 7e-6).  So every 32 instructions, 1024 k,
// the accumulator is added into fp32 registers, rounded to nearest: 1.9e-7 and 1.9e-6 at
// any depth, for 4 % of the time of a product 8192 deep and 7 % of one 4096 deep (every
// 16 instructions: 11 and 20 %).  E2M1 products are multiples of a quarter of their
// scales' product, 144 of these at most, and sums below 2^24 of the smallest quarter are
// exact: 8192 deep, whatever the signs, if the scales' products are within three powers
// of two.  They stay in the accumulator, which beyond that loses at most a unit in the
// last place per 64 k; with these joined too the prompt below took 233 us instead of 204
// (every 16 instructions 300).
//
// Bound and measured (GB300).  Few rows: HBM (64 rows over 64 experts of 2048 x 4096
// E2M1, 45 of them busy: 35 us, 5.9 TB/s, of which 5 % are the last of five rounds of
// tiles).  Many rows: no unit alone.  A k-block of 128 bytes writes 29 KB into shared
// memory, and its MMAs read 29 KB (42 KB if an SM reads both halves of X): 450 to 560
// of its 640 clocks, in which the tensor pipe is busy for 370; what the issuing thread
// does besides waiting counts in full.  32768 rows over 32 experts of 4096 x 4096, bias
// and SiLU, bf16 out: E2M1 217 to 229 us, 4.9 PFLOP/s, with new inputs each time, 205
// with the same; E4M3 401 to 410 us, 2.7 PFLOP/s.
// What there is to gain, from copies that leave work out (of a first version at 222):
// C's writes 31, W from L2 alone 21, a quarter of the MMAs 20, the scales' copies to
// tensor memory 18, X's loads 13, the scales' loads 10; without C, copies, X and scales,
// and with a quarter of the MMAs, 165 are left.
// Tried: a wait per block (212; with another for its scales 226), both blocks loaded and
// freed as one stage (219, and 16.7 against 12.8 for 777 rows over 24 experts of 1000 x
// 1056 E4M3), four stages (260), copies one block ahead of their MMAs (250 against
// 222), two pairs sharing X by multicast (214 against 203: they fit 144 of the 152
// SMs), W prefetched to L2 (208 against 210), operands without the evict-last policy
// (262 against 214), C stored evict-first, past L1 or in pairs of lanes (209 to 217
// against 212 to 214).
#include "gemm_tcgen05.cuh"
#include "grouped.cuh"
#include "mx_traits.cuh"

namespace gb300 {

namespace {

template <int ELEM>
struct MxgConfig {
    static constexpr int PAIRS = 3, STAGES = 2 * PAIRS;         // a stage holds a block; two share their scales
    static constexpr int BLOCK = 128;                           // bytes of k of a swizzled block
    static constexpr int CHUNKS = MxTraits<ELEM>::kChunks;      // 128-k scale chunks of a block
    static constexpr int A_BYTES = 128 * BLOCK, B_BYTES = kMxgMost / 2 * BLOCK, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int SFA_BYTES = 128 * 16, SF_BYTES = SFA_BYTES + 256 * 16;  // boxes of 16 scales
    static constexpr int ACC_STRIDE = kMxgMost, TMEM_COLS = 512;
    static constexpr int SF_COLS = 2 * 12 * CHUNKS, SF_SLOTS = 2;  // a pair's; W: 4 per chunk, X: 8 per chunk
    static constexpr int EPI_WARP0 = 4, EPI_WARPS = 8;
    static constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
    static constexpr int BAR_BYTES = 256, SMEM_MAX = 232448;
    // pairs of blocks (8 instructions each) summed in tensor memory before the sum moves to registers
    static constexpr bool JOINS = ELEM == kMxE4M3;
    static constexpr int SEG = JOINS ? 4 : 1 << 30;
    static_assert(2 * ACC_STRIDE + SF_SLOTS * SF_COLS <= TMEM_COLS, "accumulators and scales fit");
    static_assert((STAGES + 2 * PAIRS + 5) * 8 + 8 <= BAR_BYTES, "barriers fit their slot");
    static_assert(B_BYTES % 1024 == 0 && STAGE_BYTES % 1024 == 0, "swizzle atoms stay aligned");
    // after up to 1023 bytes of alignment: [stages][scales][barriers][group table]
    static int smem_bytes(int G) {
        return 1024 + STAGES * STAGE_BYTES + PAIRS * SF_BYTES + BAR_BYTES + (group_table_bytes(G) + 15) / 16 * 16;
    }
    static_assert(1024 + STAGES * STAGE_BYTES + PAIRS * SF_BYTES + BAR_BYTES + group_table_bytes(kMaxGroups) + 16 <=
                      SMEM_MAX, "fits the 227 KB opt-in shared memory");
};

// This cluster's tiles, in row_tile's order but in widths of steps of 16, without a division or a search per tile: a step moves `rt` and `ft` by
// fixed amounts and the group forwards.
struct MxgWalk {
    const GroupTable &table;
    int tiles_f, step_r, step_f, rt, ft, g, tiles, width;
    __device__ __forceinline__ MxgWalk(const GroupTable &t, int tiles_f_, int cluster, int nclusters)
        : table(t), tiles_f(tiles_f_), step_r(nclusters / tiles_f_), step_f(nclusters % tiles_f_),
          rt(cluster / tiles_f_), ft(cluster % tiles_f_), g(-1), tiles(t.first[t.G]), width(0) {}
    __device__ __forceinline__ bool next(GroupedTile &o) {
        if (rt >= tiles) return false;
        if (g < 0 || table.first[g + 1] <= rt) {
            do ++g;
            while (table.first[g + 1] <= rt);
            const int nt = table.first[g + 1] - table.first[g];
            width = ((table.hi[g] - table.lo[g] + nt - 1) / nt + 15) & ~15;
        }
        o.g = g;
        o.f0 = ft * 256;
        o.r0 = table.lo[g] + (rt - table.first[g]) * width;
        o.nr = min(width, table.hi[g] - o.r0);
        o.bn = (o.nr + 15) & ~15;
        rt += step_r;
        ft += step_f;
        if (ft >= tiles_f) {
            ft -= tiles_f;
            ++rt;
        }
        return true;
    }
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
    unsigned char *scales = smem + Cfg::STAGES * Cfg::STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(scales + Cfg::PAIRS * Cfg::SF_BYTES);  // (leader's) a pair's operands
                                                  // landed and both CTAs' scales laid out
    uint64_t *empty = full + Cfg::PAIRS;          // a stage's MMAs are done
    uint64_t *landed = empty + Cfg::STAGES;       // this CTA's scales of a pair have landed
    uint64_t *tfull = landed + Cfg::PAIRS;
    uint64_t *tempty = tfull + 2;
    uint64_t *mma_done = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();  // 0: leader
    const int cluster = blockIdx.x / CL, nclusters = gridDim.x / CL;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::STAGES; ++s) mbar_init(&empty[s], 1);
        for (int s = 0; s < Cfg::PAIRS; ++s) {
            mbar_init(&full[s], 1 + CL);
            mbar_init(&landed[s], 1);
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
    const uint32_t tempty0_leader = mapa_shared(smem_u32(&tempty[0]), 0);
    const uint32_t abort_local = smem_u32(const_cast<int *>(abort_flag));
    const int k_bytes = args.K / (ELEM == kMxE2M1 ? 2 : 1), blocks = (k_bytes + Cfg::BLOCK - 1) / Cfg::BLOCK;
    const int steps = (blocks + 1) / 2;  // pairs of blocks; a last one may lack its second
    MxgWalk walk(table, args.tiles_f, cluster, nclusters);
    GroupedTile t;

    if (warp == 0 || warp == 3) {
        if (lane == 0) {
            // ------------------------- TMA producers: W (warp 0), X and scales (warp 3) --
            uint32_t stage = 0, phase = 0;
            bool ok = true, issued = false;
            const uint64_t keep = l2_policy_evict_last();
            while (ok && steps > 0 && walk.next(t)) {
                const int f = t.f0 + static_cast<int>(rank) * 128;
                const int bnh = t.bn >> 1;
                const int c0 = t.r0 + static_cast<int>(rank) * bnh;  // first of this CTA's MMA columns
                const uint32_t bytes = Cfg::A_BYTES + bnh * Cfg::BLOCK;
                const int sm = t.bn <= 32 ? 0 : t.bn <= 64 ? 1 : t.bn <= 128 ? 2 : 3;  // box of 32 << sm rows' scales
                for (int b = 0; b < 2 * steps; ++b) {
                    if (!pair_wait<CL>(&empty[stage], phase ^ 1u, abort_flag, args.status, abort_local, rank)) {
                        ok = false;
                        break;
                    }
                    issued = true;
                    unsigned char *sA = smem + stage * Cfg::STAGE_BYTES;
                    const uint32_t fbar = full0_leader + 8u * (stage >> 1);
                    if (warp == 0) {
                        // (of a pair without a second block, its first alone is waited for)
                        if (rank == 0 && b % 2 == 0)
                            mbar_arrive_expect_tx(&full[stage >> 1], (b + 1 < blocks ? 4u : 2u) * bytes);
                        if (b < blocks) tma_load_3d_pair(sA, &maps.w, fbar, b * Cfg::BLOCK, f, t.g, keep);
                    } else {
                        if (b % 2 == 0) {
                            uint64_t *bar = &landed[stage / 2];
                            unsigned char *sf = scales + stage / 2 * Cfg::SF_BYTES;
                            const int box = ELEM == kMxE2M1 ? b * 8 : b / 4 * 16;  // E4M3: a pair takes half of it
                            mbar_arrive_expect_tx(bar, Cfg::SFA_BYTES + (512u << sm));
                            tma_load_3d_hint(sf, &maps.ws, bar, box, f, t.g, keep);
                            tma_load_2d_hint(sf + Cfg::SFA_BYTES, &maps.xs[sm], bar, box, t.r0, keep);
                        }
                        if (b < blocks)
                            tma_load_3d_pair(sA + Cfg::A_BYTES, &maps.x[(bnh >> 3) - 1], fbar, b * Cfg::BLOCK, c0, 0, keep);
                    }
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
            // addresses and descriptors stay in uniform registers.  A step is a pair of
            // blocks: one wait and one fence for both, and each block's stage freed by
            // itself.
            const uint64_t a_desc0 = sw128_desc(smem_u32(smem), 16u, 1024u);
            const uint64_t b_desc0 = sw128_desc(smem_u32(smem) + Cfg::A_BYTES, 16u, 1024u);
            const uint64_t sf_desc0 = plain16_desc(smem_u32(scales));
            uint32_t pair = 0, phase = 0, slot = 0;
            bool ok = true, issued = false;
            int local = 0;
            while (ok && steps > 0 && walk.next(t)) {
                const uint32_t idesc0 = mma_idesc_bs(MxTraits<ELEM>::kFmt, 256, t.bn, 0, 0);
                const bool wide = t.bn > 128;
                uint32_t acc = 0;
                for (int st = 0; st < steps; ++st) {
                    const bool opens = st % Cfg::SEG == 0, closes = st + 1 == steps || (st + 1) % Cfg::SEG == 0;
                    if (opens) {
                        acc = local & 1;
                        const uint32_t acc_phase = (local >> 1) & 1;
                        ++local;
                        ok = pair_wait<CL>(&tempty[acc], acc_phase ^ 1u, abort_flag, args.status, abort_local, rank);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                    }
                    const uint32_t d_tmem = tmem_base + acc * Cfg::ACC_STRIDE;
                    ok = pair_wait<CL>(&full[pair], phase, abort_flag, args.status, abort_local, rank);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    smem_acquire_cluster();  // the scales, written by ordinary stores
                    tc_fence_after();
                    const uint32_t at = pair * (2 * Cfg::STAGE_BYTES >> 4);  // addresses are in 16-byte units, below 2^14
                    const uint64_t ad = a_desc0 + at, bd = b_desc0 + at;
                    // E4M3: the second half of the box in odd pairs
                    const uint64_t sd = sf_desc0 + pair * (Cfg::SF_BYTES >> 4) +
                                        (ELEM == kMxE4M3 ? static_cast<uint32_t>(st & 1) * 2 * 32u : 0u);
                    // (the slot's last MMAs, two pairs back, are done: the scale warp waited for them)
                    const uint32_t sfa = tmem_base + 2 * Cfg::ACC_STRIDE + slot * Cfg::SF_COLS;
                    const uint32_t sfb = sfa + 2 * 4 * Cfg::CHUNKS;
                    const bool both = 2 * st + 1 < blocks;
                    if (elect_one()) {
#pragma unroll
                        for (int c = 0; c < 2 * Cfg::CHUNKS; ++c) {
                            if (c >= Cfg::CHUNKS && !both) break;
                            tc_cp_32x128b_x4_pair(sfa + 4 * c, sd + c * 32u);
                            tc_cp_32x128b_x4_pair(sfb + 8 * c, sd + (Cfg::SFA_BYTES >> 4) + c * 32u);
                            if (wide) tc_cp_32x128b_x4_pair(sfb + 8 * c + 4, sd + ((Cfg::SFA_BYTES + 2048) >> 4) + c * 32u);
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (h == 0 || both) {
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks) {
                                    const uint32_t chunk = Cfg::CHUNKS * h + (Cfg::CHUNKS == 1 ? 0 : ks >> 1);
                                    const uint32_t sf_id = Cfg::CHUNKS == 1 ? ks : (ks & 1) * 2;
                                    tc_mma_bs_pair<MxTraits<ELEM>::kKind>(
                                        d_tmem, ad + h * (Cfg::STAGE_BYTES >> 4) + ks * 2,
                                        bd + h * (Cfg::STAGE_BYTES >> 4) + ks * 2, idesc0 | (sf_id << 4) | (sf_id << 29),
                                        sfa + 4 * chunk, sfb + 8 * chunk, !opens || (h | ks) != 0 ? 1u : 0u);
                                }
                            }
                            tc_commit_pair(&empty[2 * pair + h], 0x3);
                        }
                        if (closes) tc_commit_pair(&tfull[acc], 0x3);
                    }
                    issued = true;
                    slot ^= 1u;
                    if (++pair == Cfg::PAIRS) {
                        pair = 0;
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
        // The issuer copies a pair's scales over those of two pairs before, and no order is promised between a copy and
        // MMAs issued earlier.  So scales are only reported once those MMAs are done (the pair's last `empty`): the
        // issuer's wait for them then covers that too.
        uint32_t pair = 0, phase = 0, old = 0, old_phase = 0;
        int ahead = 0;
        bool ok = true;
        while (ok && steps > 0 && walk.next(t)) {
            for (int st = 0; st < steps; ++st) {
                bool got = pair_wait<CL>(&landed[pair], phase, abort_flag, args.status, abort_local, rank);
                ok = __all_sync(0xffffffffu, got);
                if (!ok) break;
                const uint32_t sf = smem_u32(scales + pair * Cfg::SF_BYTES);
                lay_out_scales(sf);
                // (rows past the box are an earlier tile's scales or none: their columns are not stored)
                lay_out_scales(sf + Cfg::SFA_BYTES);
                if (t.bn > 128) lay_out_scales(sf + Cfg::SFA_BYTES + 2048);
                if (ahead < Cfg::SF_SLOTS) {
                    ++ahead;
                } else {
                    got = pair_wait<CL>(&empty[2 * old + 1], old_phase, abort_flag, args.status, abort_local, rank);
                    ok = __all_sync(0xffffffffu, got);
                    if (!ok) break;
                    if (++old == Cfg::PAIRS) {
                        old = 0;
                        old_phase ^= 1u;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    smem_release_cluster();
                    mbar_arrive_remote_relaxed(full0_leader + 8u * pair);
                }
                if (++pair == Cfg::PAIRS) {
                    pair = 0;
                    phase ^= 1u;
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
        while (walk.next(t)) {
            const int f = t.f0 + static_cast<int>(rank) * 128 + quad * 32 + lane;
            const float bias = (e.epi != kEpiNone && f < args.F)
                                   ? args.bias[static_cast<long long>(t.g) * args.F + f] : 0.0f;
            OutT *c = static_cast<OutT *>(args.C) + t.r0 * args.ldc + f;
            const float *rs = args.row_scale != nullptr ? args.row_scale + t.r0 : nullptr;
            const int chunks = (t.bn + 31) >> 5;  // (a last half chunk reads columns that are not stored)
            const int c_begin = half ? (chunks + 1) >> 1 : 0, nch = (half ? chunks : (chunks + 1) >> 1) - c_begin;
            const uint32_t t_quad = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + c_begin * 32;
            auto store = [&](float (&v)[32], int row, int nrow) {
                OutT *c0 = c + row * args.ldc;
                chunk_values_t<OUT>(v, c0, args.F - f, nrow, rs != nullptr ? rs + row : nullptr, 1.0f, bias, e);
                store_chunk_t<OUT>(v, c0, args.F - f, nrow, args.ldc);
            };
            if constexpr (Cfg::JOINS) {
                if (steps > Cfg::SEG) {
                    // halves of whole 16 columns: at most seven, 112 registers (of whole 32, 128: some spilled, 2 % slower)
                    constexpr int kMost = (kMxgMost / 16 + 1) / 2;
                    const int all = t.bn >> 4, first = half ? (all + 1) >> 1 : 0, n = (half ? all : (all + 1) >> 1) - first;
                    const uint32_t t_first = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + first * 16;
                    float sum[kMost][16];
#pragma unroll
                    for (int u = 0; u < kMost; ++u)
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[u][j] = 0.0f;
                    bool ok = true;
                    for (int st = 0; st < steps; st += Cfg::SEG) {
                        const uint32_t acc = local & 1, acc_phase = (local >> 1) & 1;
                        ++local;
                        const bool got = pair_wait<CL>(&tfull[acc], acc_phase, abort_flag, args.status, abort_local, rank);
                        ok = __all_sync(0xffffffffu, got);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int u = 0; u < kMost; ++u)
                            if (u < n) {
                                uint32_t raw[16];
                                __syncwarp();
                                tmem_ld_x16(t_first + acc * Cfg::ACC_STRIDE + u * 16, raw);
#pragma unroll
                                for (int j = 0; j < 16; ++j) sum[u][j] += __uint_as_float(raw[j]);
                            }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(tempty0_leader + 8u * acc);
                    }
                    if (!ok) break;
#pragma unroll
                    for (int u = 0; u < kMost; u += 2)
                        if (u < n) {
                            float v[32];
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = u + j / 16 < kMost ? sum[(u + j / 16) % kMost][j % 16] : 0.0f;
                            store(v, (first + u) * 16, min(t.nr - (first + u) * 16, (n - u) * 16));
                        }
                    continue;
                }
            }
            const uint32_t acc = local & 1, acc_phase = (local >> 1) & 1;
            if (steps > 0) {
                ++local;
                const bool got = pair_wait<CL>(&tfull[acc], acc_phase, abort_flag, args.status, abort_local, rank);
                if (!__all_sync(0xffffffffu, got)) break;
                tc_fence_after();
            }
#pragma unroll 1
            for (int ch = 0; ch < nch; ++ch) {
                float v[32];
                if (steps > 0) {
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
                if (steps > 0 && ch + 1 == nch) {
                    // the accumulator is in registers: free it before the stores
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(tempty0_leader + 8u * acc);
                }
                const int row = (c_begin + ch) * 32;
                store(v, row, t.nr - row);
            }
            if (steps > 0 && nch == 0) {  // a tile of up to 32 columns has no second half
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
