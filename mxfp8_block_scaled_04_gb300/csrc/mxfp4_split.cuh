// MXFP4 products with few tiles: one 128 x 128 tile per CTA or, with a cluster of S CTAs, per cluster, each CTA taking
// a share of K; the partial sums meet through distributed shared memory and are added in rank order.
//
// Two CTAs fit an SM, so one's start and end overlap the other's loads, and every tile of a wide layer is
// resident at once: at one token the weights' bytes are the time, and all CTAs share HBM evenly whatever the
// tiles' number.  Roles as in mxfp4_gemm.cuh.
//
// Measured: 1x8192x28672 22.0 us (125 MB of weights, 5.7 TB/s), 1x4096x4096 5.6 us (K in eight parts),
// 1x8192x8192 9.1 us; 333x4096x4096 about 9 us.  What is left over the bytes is the start and end of the CTAs.
#pragma once

#include "mxfp4_gemm.cuh"

namespace mxfp8 {

// QROWS: rows of Q that the stages hold.  Two CTAs fit an SM with 4 stages of 32 rows or 3 of 128.  (The occupancy
// query reports one for any kernel that allocates TMEM; CTAs of 256 columns were seen to run side by side.)
template <int QROWS, int STAGES>
struct SplitShape {
    static constexpr int kPBytes = kGemmRows * 128;
    static constexpr int kQBytes = QROWS * 128;
    static constexpr int kStage = kPBytes + kQBytes + 2048;  // + two scale tiles of each operand
    static constexpr int kStages = STAGES;
    static constexpr int kSmem = kStages * kStage + 1024;
    static constexpr int kColumns = 256;                     // TMEM: accumulator at 0, scales at 128
};

__device__ __forceinline__ float4 load_peer(uint32_t mapped)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(mapped) : "memory");
    return v;
}

template <int QROWS, int STAGES, bool F32, int PARTS>
__global__ void __launch_bounds__(kGemmThreads, 2)
    mxfp4_split_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map, const GemmParams p, int splits)
{
    using S = SplitShape<QROWS, STAGES>;
    extern __shared__ unsigned char gemm_smem[];
    __shared__ uint64_t full[S::kStages], empty[S::kStages], acc_full, drain;
    __shared__ uint32_t tmem_slot;

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const uint32_t base = (smem_u32(gemm_smem) + 1023u) & ~1023u;
    unsigned char *smem = gemm_smem + (base - smem_u32(gemm_smem));
    if (tid == 0) {
        prefetch_tensormap(&p_map);
        prefetch_tensormap(&q_map);
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 2);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(&acc_full), 1);
        mbar_init(smem_u32(&drain), 1);
        fence_mbar_init();
    }
    if (warp == 2)
        tmem_alloc(smem_u32(&tmem_slot), S::kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    if constexpr (PARTS == 1)
        pdl_wait_and_release();

    const int rank = static_cast<int>(blockIdx.x) % splits;
    const GemmTile c = gemm_tile<kGemmRows, 128, false>(static_cast<int>(blockIdx.x) / splits, p, GroupTable<false>{});
    const int k0 = static_cast<int>(static_cast<int64_t>(p.k_iters) * rank / splits);
    const int k1 = static_cast<int>(static_cast<int64_t>(p.k_iters) * (rank + 1) / splits);
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
    // With parts, the kernel before on the stream writes Q alone, and began after all before it had ended: the weights of the
    // first stages are loaded while it runs (1x8192x8192 11.3 -> 10.3 us, 1x8192x28672 24.2 -> 23.0).
    const int early = PARTS > 1 ? min(S::kStages, k1 - k0) : 0;
    if constexpr (PARTS > 1) {
        if (warp == 0 || warp == 3) {
            const int boxes = (c.valid + p.q_box - 1) / p.q_box;
            for (int j = 0; j < early; ++j) {
                if (elect_one()) {
                    const uint32_t bar = full0 + 8 * j, dp = base + j * S::kStage;
                    if (warp == 0) {
                        mbar_arrive_expect_tx(bar, S::kPBytes + boxes * p.q_box * 128);
                        tma_load_2d_shared(dp, &p_map, bar, (k0 + j) * 128, c.p_row);
                    } else {
                        const uint32_t sb = 512u * min(2, p.kc - 2 * (k0 + j));
                        mbar_arrive_expect_tx(bar, 2 * sb);
                        bulk_load(dp + S::kPBytes + S::kQBytes, p.p_scale + c.p_plane * p.kc * 512 + int64_t{k0 + j} * 1024, sb, bar);
                    }
                }
                __syncwarp();
            }
        }
        pdl_wait_and_release();
    }

    if (warp == 0 || warp == 3) {
        // ---- producers: codes (warp 0), scales (warp 3) ----
        const int boxes = (c.valid + p.q_box - 1) / p.q_box;
        const uint32_t code_bytes = S::kPBytes + boxes * p.q_box * 128;
        const uint8_t *ps = p.p_scale + c.p_plane * p.kc * 512, *qs = p.q_scale + c.q_plane * p.kc * 512;
        int issued = 0;
        for (int k = k0; k < k1; ++k) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_cycles(empty0 + 8 * slot, phase ^ 1, kGemmWait));
            if (!ok)
                break;
            const uint32_t bar = full0 + 8 * slot, dp = base + slot * S::kStage;
            const bool started = k - k0 < early;  // its weights are on their way
            if (elect_one()) {
                if (warp == 0) {
                    if (!started) {
                        mbar_arrive_expect_tx(bar, code_bytes);
                        tma_load_2d_shared(dp, &p_map, bar, k * 128, c.p_row);
                    }
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d_shared(dp + S::kPBytes + b * p.q_box * 128, &q_map, bar, k * 128, c.q_row + b * p.q_box);
                } else {
                    const uint32_t sb = 512u * min(2, p.kc - 2 * k), ds = dp + S::kPBytes + S::kQBytes;
                    if (!started) {
                        mbar_arrive_expect_tx(bar, 2 * sb);
                        bulk_load(ds, ps + int64_t{k} * 1024, sb, bar);
                    }
                    bulk_load(ds + 1024, qs + int64_t{k} * 1024, sb, bar);
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
        const int n = (c.valid + 15) & ~15;
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
        // ---- this CTA's sums: to the output, or to shared memory for the cluster (every stage has been consumed) ----
        const int quarter = warp & 3;
        ok = epilogue_all(mbar_wait_cycles(smem_u32(&acc_full), 0, kGemmWait));
        if (ok) {
            tc_fence_after();
            for (int q = 0; q < c.valid; q += 32) {
                uint32_t v[32];
                tmem_load32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + q, v);
                if (splits == 1) {
                    if constexpr (PARTS > 1)
                        store_parts<F32, PARTS>(p, v, quarter, lane, c.q_row + q, c.valid - q, c.p0);
                    else
                        store_chunk<F32>(p, v, smem + (q & 32 ? kEpiBytes<F32> / 2 : 0), quarter, lane, c.q_row + q, c.valid - q, c.p0);
                } else if constexpr (PARTS > 1) {  // the parts of a row are added here, the smallest first
                    float *part = reinterpret_cast<float *>(smem) + q / PARTS * kGemmRows + quarter * 32 + lane;
#pragma unroll
                    for (int t = 0; t < 32 / PARTS; ++t) {
                        float sum = __uint_as_float(v[PARTS * t + PARTS - 1]);
#pragma unroll
                        for (int j = PARTS - 2; j >= 0; --j)
                            sum += __uint_as_float(v[PARTS * t + j]);
                        if (q + PARTS * t < c.valid)
                            part[t * kGemmRows] = sum;
                    }
                } else {
                    float *part = reinterpret_cast<float *>(smem) + q * kGemmRows + quarter * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (q + j < c.valid)
                            part[j * kGemmRows] = __uint_as_float(v[j]);
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
    if (splits > 1) {
        cluster_sync();
        for (int i = rank * kGemmThreads + tid; i < c.valid / PARTS * (kGemmRows / 4); i += splits * kGemmThreads) {
            const int row = i / (kGemmRows / 4), col = i % (kGemmRows / 4) * 4;
            const uint32_t at = base + i * 16;
            float4 sum = load_peer(map_to_rank(at, 0));
            for (int r = 1; r < splits; ++r) {
                const float4 v = load_peer(map_to_rank(at, r));
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
            const int64_t to = (int64_t{c.q_row} / PARTS + row) * p.ldo + c.p0 + col;
            if (p.vec_out) {
                if (c.p0 + col < p.P) {
                    if constexpr (F32)
                        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + to) = sum;
                    else
                        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + to) =
                            make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
                }
            } else {
                const float s[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c.p0 + col + j < p.P)
                        store_out<F32>(p.out, to + j, __float_as_uint(s[j]));
            }
        }
        cluster_sync();  // the peers have read this CTA's sums
    }
}

}  // namespace mxfp8
