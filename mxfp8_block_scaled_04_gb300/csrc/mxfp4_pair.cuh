// MXFP4 products in tiles of 256 x 256 by pairs of CTAs (cta_group::2): the kernel for many rows.
//
// Each CTA of a pair keeps 128 rows of P and half of Q's 256 rows in shared memory and 128 lanes x 256 columns of
// the accumulator in TMEM; the first CTA's MMA warp issues for both.  Against 128 x 128 tiles of one CTA this halves
// the operand bytes per product (8192x8192x28672: 824 -> 603 us).  Two accumulators of 256 columns and the scales do
// not fit TMEM's 512 columns side by side, so the accumulators share 32 columns: the epilogue drains those first
// and the next tile's MMAs begin while it drains the rest.  Output rows leave as 16-byte pieces (603 -> 511 us).
//
// Measured: 8192x8192x28672 490 us alone (7.9 PFLOP/s), about 570 us back to back under the power limit.  Bound by the
// MMAs: without the output, Q's loads and the scale copies the same loop takes 461 us; the tensor pipe is active
// 74% of the cycles at 4096x8192x8192 (seven rounds of tiles); three, four and five stages take the same time.
//
// TMEM columns: accumulator 0 at 0, accumulator 1 at 224, scales at 480 (per half stage: 4 for P, 8 for Q).
#pragma once

#include "mxfp4_gemm.cuh"

namespace mxfp8 {

constexpr int kPairRows = 256;                    // rows of P, and of Q, per tile
constexpr int kPairStages = 5;
constexpr int kPairCodes = 128 * 128;             // bytes of either operand's rows in one CTA
constexpr int kPairPScale = 1024, kPairQScale = 2048;
constexpr int kPairStage = 2 * kPairCodes + kPairPScale + kPairQScale;
constexpr int kPairSmem = kPairStages * kPairStage + 1024;  // + the epilogue's buffers
constexpr int kPairAcc1 = 224, kPairShared = 32, kPairScaleCol = 480;

template <bool F32, bool GROUPED>
__global__ void __launch_bounds__(kGemmThreads, 1)
    mxfp4_pair_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap q_part_map, const __grid_constant__ CUtensorMap ps_map, const __grid_constant__ CUtensorMap qs_map, const GemmParams p)
{
    extern __shared__ unsigned char gemm_smem[];
    __shared__ GroupTable<GROUPED> groups;
    __shared__ uint64_t full[kPairStages], empty[kPairStages], acc_full[2], acc_empty, drain;
    __shared__ uint32_t tmem_slot;

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const uint32_t rank = cluster_rank();
    const uint32_t base = (smem_u32(gemm_smem) + 1023u) & ~1023u;
    if (tid == 0) {
        prefetch_tensormap(&p_map);
        prefetch_tensormap(&q_map);
        prefetch_tensormap(&q_part_map);
        prefetch_tensormap(&ps_map);
        prefetch_tensormap(&qs_map);
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(&acc_full[0]), 1);
        mbar_init(smem_u32(&acc_full[1]), 1);
        mbar_init(smem_u32(&acc_empty), 8);  // the epilogue warps of both CTAs
        mbar_init(smem_u32(&drain), 1);
        fence_mbar_init();
    }
    if (warp == 2)
        tmem_alloc_pair(smem_u32(&tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait_and_release();

    int num_tiles = p.p_tiles * p.q_tiles;
    int64_t no_expert = p.Q;  // the first row of no expert
    if constexpr (GROUPED) {
        const int rt = group_setup<kGemmThreads, kPairRows>(groups, p.offsets, p.num_groups, p.Q);
        num_tiles = rt < 0 ? 0 : rt * p.p_tiles;
        if (rt >= 0)
            no_expert = groups.offset[p.num_groups];
        if (blockIdx.x == 0 && tid == 0 && p.err_flag != nullptr && (rt < 0 || no_expert < p.Q))
            atomicOr(p.err_flag, 1);
    }
    // The pair's n-th tile: rounds of one tile per pair, every other one backwards, so that a partial last round goes to
    // the pairs whose tiles in the round before came last (4099 rows: the 3-row tiles, not whole ones).
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    auto tile_of = [&](int n) { return n * pairs + (n & 1 ? pairs - 1 - pair : pair); };
    const uint32_t full0 = smem_u32(&full[0]), empty0 = smem_u32(&empty[0]);
    int slot = 0;
    uint32_t phase = 0;
    auto advance = [&]() {
        if (++slot == kPairStages) {
            slot = 0;
            phase ^= 1;
        }
    };

    if (warp == 0 || warp == 3) {
        // ---- producers of this CTA's operands: codes (warp 0), scales (warp 3); they signal the first CTA's barriers ----
        const uint32_t lead_full = map_to_rank(full0, 0);
        bool ok = true;
        int issued = 0;
        for (int n = 0, t; (t = tile_of(n)) < num_tiles && ok; ++n) {
            const GemmTile c = gemm_tile<kPairRows, kPairRows, GROUPED>(t, p, groups);
            const int half = ((c.valid + 31) & ~31) / 2;
            const int boxes = half > 96 ? 0 : (half + 31) / 32;  // a partial tile's rows of Q in boxes of 32 (0: whole)
            const uint32_t bytes = 2 * (kPairStage - (boxes ? (4 - boxes) * 32 * 128 : 0));  // of both CTAs
            for (int k = 0; k < p.k_iters; ++k) {
                ok = mbar_wait_cluster(empty0 + 8 * slot, phase ^ 1, kGemmWait);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = lead_full + 8 * slot, dp = base + slot * kPairStage;
                if (elect_one()) {
                    if (warp == 0) {
                        if (rank == 0)
                            mbar_arrive_expect_tx(full0 + 8 * slot, bytes);
                        tma_load_2d_pair(dp, &p_map, bar, k * 128, c.p_row + static_cast<int>(rank) * 128);
                        if (boxes == 0)
                            tma_load_2d_pair(dp + kPairCodes, &q_map, bar, k * 128, c.q_row + static_cast<int>(rank) * half);
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d_pair(dp + kPairCodes + b * 32 * 128, &q_part_map, bar, k * 128, c.q_row + static_cast<int>(rank) * half + 32 * b);
                    } else {
                        const uint32_t ds = dp + 2 * kPairCodes;
                        tma_load_2d_pair(ds, &ps_map, bar, k * 256, static_cast<int>(c.p_plane) + static_cast<int>(rank));
                        tma_load_2d_pair(ds + kPairPScale, &qs_map, bar, k * 256, static_cast<int>(c.q_plane));
                    }
                }
                __syncwarp();
                ++issued;
                advance();
            }
        }
        if (!ok && lane == 0)
            atomicOr(p.fault, 1u);
        if (rank == 0 && !ok) {
            for (int j = 0; j < kPairStages && j < issued; ++j) {  // copies in flight, the newest first
                if (--slot < 0) {
                    slot = kPairStages - 1;
                    phase ^= 1;
                }
                mbar_wait_cluster(full0 + 8 * slot, phase, kGemmDrain);
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---- MMA for both CTAs ----
        bool ok = true;
        const uint64_t p_desc = desc_sw128(base), q_desc = desc_sw128(base + kPairCodes);
        const uint64_t s_desc = desc_scales(base + 2 * kPairCodes);
        for (int n_tile = 0, t; (t = tile_of(n_tile)) < num_tiles && ok; ++n_tile) {
            const GemmTile c = gemm_tile<kPairRows, kPairRows, GROUPED>(t, p, groups);
            const int n = (c.valid + 31) & ~31;  // halves of whole 16-row groups
            const uint32_t d = tmem + (n_tile & 1) * kPairAcc1, sf = tmem + kPairScaleCol;
            const uint32_t idesc0 = mxf4_idesc(kPairRows, n, 0), idesc1 = mxf4_idesc(kPairRows, n, 1);
            if (n_tile >= 1)  // the columns shared with the tile before are read, and all of the one before that
                ok = mbar_wait_cluster(smem_u32(&acc_empty), (n_tile - 1) & 1, kGemmWait);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            for (int k = 0; k < p.k_iters; ++k) {
                ok = mbar_wait_cluster(full0 + 8 * slot, phase, kGemmWait);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t step = slot * (kPairStage >> 4);
                    const uint64_t pd = p_desc + step, qd = q_desc + step, sd = s_desc + step;
                    const int left = p.k64 - 4 * k;
#pragma unroll
                    for (int ch = 0; ch < 2; ++ch) {
                        if (left <= 2 * ch)
                            break;
                        const uint32_t sp = sf + ch * 12, sq = sp + 4;
                        tc_copy_scales_pair(sp, sd + ch * 32);
                        tc_copy_scales_pair(sq, sd + (kPairPScale + ch * 512) / 16);
                        tc_copy_scales_pair(sq + 4, sd + (kPairPScale + 1024 + ch * 512) / 16);
                        tc_mma_mxf4_pair(d, pd + ch * 4, qd + ch * 4, idesc0, sp, sq, k > 0 || ch > 0);
                        if (left > 2 * ch + 1)
                            tc_mma_mxf4_pair(d, pd + ch * 4 + 2, qd + ch * 4 + 2, idesc1, sp, sq, true);
                    }
                    tc_commit_pair(empty0 + 8 * slot);
                    if (k == p.k_iters - 1)
                        tc_commit_pair(smem_u32(&acc_full[n_tile & 1]));
                }
                __syncwarp();
                advance();
            }
        }
        if (!ok) {
            if (elect_one()) {
                atomicOr(p.fault, 1u);
                tc_commit_pair(smem_u32(&drain));
            }
            __syncwarp();
            mbar_wait_cluster(smem_u32(&drain), 0, kGemmDrain);
        }
    } else if (warp >= 4) {
        // ---- epilogue of this CTA's 128 columns of the output ----
        const int quarter = warp & 3;
        const uint32_t lead_empty = map_to_rank(smem_u32(&acc_empty), 0);
        unsigned char *stage_out = gemm_smem + (base - smem_u32(gemm_smem)) + kPairStages * kPairStage;
        int chunk = 0;
        if constexpr (GROUPED)
            clear_rows_from<F32>(p, no_expert, quarter * 32 + lane);
        for (int n_tile = 0, t; (t = tile_of(n_tile)) < num_tiles; ++n_tile) {
            const GemmTile c = gemm_tile<kPairRows, kPairRows, GROUPED>(t, p, groups);
            const int buf = n_tile & 1;
            if (!epilogue_all(mbar_wait_cluster(smem_u32(&acc_full[buf]), (n_tile >> 1) & 1, kGemmWait))) {
                if (lane == 0)
                    atomicOr(p.fault, 1u);
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * kPairAcc1;
            // the columns shared with the other accumulator first: 224..255 of accumulator 0, 0..31 of accumulator 1
            const int start = buf == 0 ? kPairAcc1 : 0;
            for (int i = 0; i < kPairRows / 32; ++i) {
                const int q = (start + 32 * i) & (kPairRows - 1);
                uint32_t v[32];
                if (q < c.valid)
                    tmem_load32(d + q, v);
                if (i == 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster(lead_empty);
                }
                if (q < c.valid)
                    store_chunk<F32>(p, v, stage_out + (chunk++ & 1) * (kEpiBytes<F32> / 2), quarter, lane, c.q_row + q, c.valid - q,
                                     c.p0 + rank * 128);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its pair's MMAs, copies or arrivals may still reach it
    if (warp == 2)
        tmem_dealloc_pair(tmem, 512);
}

}  // namespace mxfp8
