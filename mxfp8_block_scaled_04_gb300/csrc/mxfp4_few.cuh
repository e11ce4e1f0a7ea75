// Up to kFewRows uncast rows on 4-bit weights in one launch: the product of mxfp4_split.cuh, whose CTAs split x into the parts
// of mxfp4_parts.cuh themselves, straight into the operand's shared memory.
//
// While the weights stream in, the four epilogue warps have nothing else to do: each in turn makes a stage's 256 columns of
// two rows, eight parts of 8 columns per lane and row, and arrives on the stage's barrier with the copies.  Every CTA repeats this for
// its share of K; against a kernel of its own that writes the parts, a launch, its gap and the workspace fall away.
// 1x8192x28672 in 20.9 us (6.0 TB/s), 1x4096x4096 in 5.1.  Bound by the weights' bytes, or the start and end of the CTAs; more rows
// by the splitting, whose four warps issue too little (few_rows() in mxfp4.cu has the limit).
//
// Experts: a tile is 128 columns of one row, whose expert the CTA finds in the offsets, which it checks itself.  Rows that share an
// expert read its weights again, through L2 (few_expert_rows() has the limit).
#pragma once

#include "mxfp4_parts.cuh"
#include "mxfp4_split.cuh"

namespace mxfp8 {

constexpr int kFewRows = 8;

// MROWS: rows of x that the stages hold (2, 4 or 8).
template <int MROWS, int STAGES, bool XF32, bool F32, bool GROUPED>
__global__ void __launch_bounds__(kGemmThreads, 2)
    mxfp4_few_kernel(const __grid_constant__ CUtensorMap p_map, const GemmParams p, const PartsParams x, int splits)
{
    using S = SplitShape<MROWS * kParts, STAGES>;
    extern __shared__ unsigned char gemm_smem[];
    __shared__ uint64_t full[S::kStages], empty[S::kStages], acc_full, drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int expert;

    const int rows = GROUPED ? 1 : static_cast<int>(x.R), pairs = (rows + 1) / 2;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const uint32_t base = (smem_u32(gemm_smem) + 1023u) & ~1023u;
    unsigned char *smem = gemm_smem + (base - smem_u32(gemm_smem));
    if (tid == 0) {
        prefetch_tensormap(&p_map);
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 2 + pairs);  // the weights' codes and scales, each two rows
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(&acc_full), 1);
        mbar_init(smem_u32(&drain), 1);
        expert = -1;
        fence_mbar_init();
    }
    if (warp == 2)
        tmem_alloc(smem_u32(&tmem_slot), S::kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait_and_release();

    const int rank = static_cast<int>(blockIdx.x) % splits;
    int tile = static_cast<int>(blockIdx.x) / splits, p_row = 0;
    int64_t from = 0, to = 0;  // x's first row, the output's
    bool live = true, idle = false;  // live: `from` is a row of x; idle: nothing to add up (a cluster's CTAs agree)
    const uint8_t *ps = p.p_scale;
    if constexpr (GROUPED) {
        to = tile / p.p_tiles;
        tile -= static_cast<int>(to) * p.p_tiles;
        int bad = tid == 0 && p.offsets[0] != 0;
        for (int g = tid; g < p.num_groups; g += kGemmThreads) {
            const int64_t a = p.offsets[g], b = p.offsets[g + 1];
            bad |= a < 0 || b < a || b > x.R;
            if (a <= to && to < b)
                expert = g;  // (of bad offsets perhaps one of several: it is not used)
        }
        bad = __syncthreads_or(bad);
        from = x.rows != nullptr ? x.rows[to] : to;
        idle = bad || expert < 0;
        // a row of no expert is one that a plan marks as such, or lost
        live = from >= 0 && from < x.T;
        if (blockIdx.x % (p.p_tiles * splits) == 0 && tid == 0 && p.err_flag != nullptr && (bad || (expert < 0 ? x.rows == nullptr || from >= 0 : !live)))
            atomicOr(p.err_flag, 1);
        if (!bad && expert < 0 && rank == 0 && tid < kGemmRows && tile * int64_t{kGemmRows} + tid < p.P)
            store_out<F32>(p.out, to * p.ldo + tile * int64_t{kGemmRows} + tid, 0u);
        if (!idle) {
            p_row = static_cast<int>(expert * p.P);
            ps += static_cast<int64_t>(expert) * p.p_planes * p.kc * 512;
        }
    }
    const int64_t p0 = static_cast<int64_t>(tile) * kGemmRows;
    ps += static_cast<int64_t>(tile) * p.kc * 512;
    const int k0 = static_cast<int>(static_cast<int64_t>(p.k_iters) * rank / splits);
    const int k1 = idle ? k0 : static_cast<int>(static_cast<int64_t>(p.k_iters) * (rank + 1) / splits);
    const uint32_t full0 = smem_u32(&full[0]), empty0 = smem_u32(&empty[0]);
    int slot = 0;
    uint32_t phase = 0;
    auto advance = [&]() {
        if (++slot == S::kStages) {
            slot = 0;
            phase ^= 1;
        }
    };
    bool ok = true;

    if (warp == 0 || warp == 3) {
        // ---- producers of the weights: codes (warp 0), scales (warp 3) ----
        int issued = 0;
        for (int k = k0; k < k1; ++k) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_cycles(empty0 + 8 * slot, phase ^ 1, kGemmWait));
            if (!ok)
                break;
            const uint32_t bar = full0 + 8 * slot, dp = base + slot * S::kStage;
            if (elect_one()) {
                if (warp == 0) {
                    mbar_arrive_expect_tx(bar, S::kPBytes);
                    tma_load_2d_shared(dp, &p_map, bar, k * 128, p_row + static_cast<int>(p0));
                } else {
                    const uint32_t sb = 512u * min(2, p.kc - 2 * k);
                    mbar_arrive_expect_tx(bar, sb);
                    bulk_load(dp + S::kPBytes + S::kQBytes, ps + int64_t{k} * 1024, sb, bar);
                }
            }
            __syncwarp();
            ++issued;
            advance();
        }
        if (!ok) {
            for (int j = 0; j < S::kStages && j < issued; ++j) {  // copies in flight, the newest first
                if (--slot < 0) {
                    slot = S::kStages - 1;
                    phase ^= 1;
                }
                mbar_wait_cycles(full0 + 8 * slot, phase, kGemmDrain);
            }
        }
    } else if (warp == 1) {
        // ---- MMA ----
        const uint64_t p_desc = desc_sw128(base), q_desc = desc_sw128(base + S::kPBytes);
        const uint64_t s_desc = desc_scales(base + S::kPBytes + S::kQBytes);
        const int n = (rows * kParts + 15) & ~15;  // (the columns past the rows' hold what the memory held)
        const uint32_t idesc0 = mxf4_idesc(kGemmRows, n, 0), idesc1 = mxf4_idesc(kGemmRows, n, 1);
        for (int k = k0; k < k1; ++k) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_cycles(full0 + 8 * slot, phase, kGemmWait));
            if (!ok)
                break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t step = slot * (S::kStage >> 4);
                const uint64_t pd = p_desc + step, qd = q_desc + step, sd = s_desc + step;
                const int left = p.k64 - 4 * k;
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    if (left <= 2 * ch)
                        break;
                    const uint32_t sp = tmem + 128 + ch * 8, sq = sp + 4;
                    tc_copy_scales(sp, sd + ch * 32);
                    tc_copy_scales(sq, sd + (1024 + ch * 512) / 16);
                    tc_mma_mxf4(tmem, pd + ch * 4, qd + ch * 4, idesc0, sp, sq, k > k0 || ch > 0);
                    if (left > 2 * ch + 1)
                        tc_mma_mxf4(tmem, pd + ch * 4 + 2, qd + ch * 4 + 2, idesc1, sp, sq, true);
                }
                tc_commit(empty0 + 8 * slot);
                if (k == k1 - 1)
                    tc_commit(smem_u32(&acc_full));
            }
            __syncwarp();
            advance();
        }
        if (!ok) {
            if (elect_one())
                tc_commit(smem_u32(&drain));
            __syncwarp();
            mbar_wait_cycles(smem_u32(&drain), 0, kGemmDrain);
        }
    } else if (warp >= 4) {
        // ---- the rows' parts: two rows of a stage at a time in turn to these four warps ----
        const int quarter = warp & 3, tasks = (k1 - k0) * pairs;
        struct Piece {
            uint4 lo, hi;
        };
        Piece next[2];
        auto fetch = [&](int t) {  // a task's columns, loaded while the warp's one before it is split
            const int it = t / pairs, m0 = 2 * (t - it * pairs);
            const int64_t c = static_cast<int64_t>(k0 + it) * 256 + lane * 8;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                next[i] = Piece{};
                if (m0 + i < rows && t < tasks && c < x.K && live) {  // K is a multiple of 8
                    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(x.x) + ((from + m0 + i) * x.ldx + c) * (XF32 ? 4 : 2));
                    next[i].lo = src[0];
                    if constexpr (XF32)
                        next[i].hi = src[1];
                }
            }
        };
        fetch(quarter);
        for (int t = quarter; t < tasks; t += 4) {
            const int it = t / pairs, m0 = 2 * (t - it * pairs), s = it % S::kStages;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_cycles(empty0 + 8 * s, ((it / S::kStages) & 1) ^ 1, kGemmWait));
            if (!ok)
                break;
            unsigned char *codes = smem + s * S::kStage + S::kPBytes + m0 * 1024 + (lane & 3) * 4;
            // row 8m of the scale tile of the lane's four blocks
            unsigned char *scale = smem + s * S::kStage + S::kPBytes + S::kQBytes + 1024 + (lane >> 4) * 512 + (8 * m0 % 32) * 16 + 8 * m0 / 32 * 4;
            const Piece at[2] = {next[0], next[1]};
            fetch(t + 4);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v[8];
                if constexpr (XF32) {
                    const uint32_t w[8] = {at[i].lo.x, at[i].lo.y, at[i].lo.z, at[i].lo.w, at[i].hi.x, at[i].hi.y, at[i].hi.z, at[i].hi.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = __uint_as_float(w[j]);
                } else {
                    const uint32_t w[4] = {at[i].lo.x, at[i].lo.y, at[i].lo.z, at[i].lo.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[2 * j] = bf16_lo(w[j]);
                        v[2 * j + 1] = bf16_hi(w[j]);
                    }
                }
                if (m0 + i < rows)
                    split_parts(v, live, [&](int j, uint32_t q, uint32_t scales) {
                        *reinterpret_cast<uint32_t *>(codes + i * 1024 + j * 128 + (((lane >> 2) ^ j) << 4)) = q;
                        if ((lane & 15) == 0)
                            *reinterpret_cast<uint32_t *>(scale + (8 * i + j) * 16) = scales;
                    });
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(full0 + 8 * s);
        }
        // ---- this CTA's sums: to the output, or to shared memory for the cluster (every stage has been consumed) ----
        if (!idle)
            ok = epilogue_all(ok && mbar_wait_cycles(smem_u32(&acc_full), 0, kGemmWait));
        if (ok && !idle) {
            tc_fence_after();
            const int valid = rows * kParts;
            for (int q = 0; q < valid; q += 32) {
                uint32_t v[32];
                tmem_load32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + q, v);
                if (splits == 1) {
                    store_parts<F32, kParts>(p, v, quarter, lane, to * kParts + q, valid - q, p0);
                } else {
                    float *part = reinterpret_cast<float *>(smem) + q / kParts * kGemmRows + quarter * 32 + lane;
#pragma unroll
                    for (int t = 0; t < 32 / kParts; ++t) {
                        float sum = __uint_as_float(v[kParts * t + kParts - 1]);
#pragma unroll
                        for (int j = kParts - 2; j >= 0; --j)
                            sum += __uint_as_float(v[kParts * t + j]);
                        if (q + kParts * t < valid)
                            part[t * kGemmRows] = sum;
                    }
                }
            }
        }
    }
    if (!ok && lane == 0)
        atomicOr(p.fault, 1u);
    tc_fence_before();
    __syncthreads();
    if (warp == 2)
        tmem_dealloc(tmem, S::kColumns);
    if (splits > 1 && !idle) {
        cluster_sync();
        for (int i = rank * kGemmThreads + tid; i < rows * (kGemmRows / 4); i += splits * kGemmThreads) {
            const int row = i / (kGemmRows / 4), col = i % (kGemmRows / 4) * 4;
            const uint32_t at = base + i * 16;
            float4 sum = load_peer(map_to_rank(at, 0));
            for (int r = 1; r < splits; ++r) {
                const float4 v = load_peer(map_to_rank(at, r));
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
            const float s[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (p0 + col + j < p.P)
                    store_out<F32>(p.out, (to + row) * p.ldo + p0 + col + j, __float_as_uint(s[j]));
        }
        cluster_sync();  // the peers have read this CTA's sums
    }
}

}  // namespace mxfp8
