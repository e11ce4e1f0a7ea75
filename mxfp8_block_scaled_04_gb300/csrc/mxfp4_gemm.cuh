// MXFP4 products on the tensor cores (sm_103a): out[q, p] = sum_k Q[q, k] * P[p, k].  What the three kernels share,
// and the experts' kernel for few rows per expert.
//
// P (a layer's weights) takes the accumulator's lanes and Q (the tokens) its columns, so that a warp writes
// neighbouring elements of an output row and the MMA's n shrinks with the tokens: the same layout serves a single
// token and a training batch.  Each block of 32 is scaled inside the MMA (kind::mxf4, two E8M0 scales per 64
// elements), so the operands go from HBM to the tensor core as they are stored; products are exact, sums fp32.
//
//   mxfp4_pair.cuh    many rows: 256 x 256 tiles by CTA pairs, bound by the tensor cores
//   mxfp4_split.cuh   few tiles: one per CTA, or K shared by a cluster, bound by the weights' bytes
//   mxfp4_group_kernel (below)   experts with few rows each: persistent 128 x 128 tiles, bound by the weights' bytes
//                     (128 rows over 64 experts of 2048 x 7168: 67 us, 6.5 TB/s; 80 cold)
//
// Roles of a CTA (8 warps): warps 0 and 3 feed a ring of shared-memory stages of 256 elements of K (TMA tiles of the
// codes; the scale tiles), warp 1 copies scales to TMEM and issues the MMAs, warp 2 owns the TMEM allocation, warps
// 4-7 read the accumulators and write the output, here while the next tile accumulates in the other TMEM buffer.
// The issuing warps run as whole warps and elect a lane per issue: from one diverged lane the issue itself bound every
// stage (8192x8192x28672: 2018 us against 824 with this change alone).  Every wait is bounded: on expiry the CTA sets
// the library's fault word, waits (bounded) for its own copies and MMAs, frees its TMEM and returns.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "groups.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace mxfp8 {

constexpr int kGemmThreads = 256;
constexpr int kGemmRows = 128;   // rows of P per tile
constexpr int64_t kGemmWait = 4000000000;   // cycles: about 2 s
constexpr int64_t kGemmDrain = 400000000;

struct GemmParams {
    const uint8_t *p_scale, *q_scale;
    int64_t P, Q;        // rows of each operand (P of one expert when grouped)
    int kc;              // scale tiles along K: ceil(K / 128)
    int k_iters;         // stages along K: ceil(K / 256)
    int k64;             // MMA steps along K: ceil(K / 64)
    int p_tiles, q_tiles;
    int p_planes;        // 128-row scale tiles of P (of one expert)
    int q_box;           // rows of Q per TMA box
    void *out;
    int64_t ldo;
    bool vec_out;        // output rows are whole 16-byte vectors
    unsigned *fault;
    const int64_t *offsets;  // grouped
    int num_groups;
    int *err_flag;
};

// The experts' kernel: 128 rows of either operand per stage, two 512-byte scale tiles each.
constexpr int kGroupBytes = kGemmRows * 128;
constexpr int kGroupStage = 2 * kGroupBytes + 2048;
constexpr int kGroupStages = 5;
constexpr int kGroupSmem = kGroupStages * kGroupStage + 1024;  // + the epilogue's buffers
constexpr int kGroupScaleCol = 256;                            // TMEM: accumulators at 0 and 128, scales from here

struct GemmTile {
    int32_t p_row, q_row;      // TMA rows
    int64_t p_plane, q_plane;  // scale tile rows
    int64_t p0;                // first output column
    int valid;                 // rows of Q in the tile
};

// Tile t.  Dense: bands of 8 Q tiles, P tiles in turn within a band, so that the CTAs at work share operands in
// L2.  Grouped: an expert's Q tiles in turn, each over all of the expert's P tiles.
template <int PT, int QT, bool GROUPED>
__device__ __forceinline__ GemmTile gemm_tile(int t, const GemmParams &p, const GroupTable<GROUPED> &groups)
{
    GemmTile r;
    if constexpr (GROUPED) {
        const int rt = t / p.p_tiles, pt = t - rt * p.p_tiles;
        const int g = groups.find(rt, p.num_groups);
        const int local = rt - groups.tile[g];
        const int64_t q0 = groups.offset[g] + static_cast<int64_t>(local) * QT;
        const int64_t left = groups.offset[g + 1] - q0;
        r.valid = left < QT ? static_cast<int>(left) : QT;
        r.q_row = static_cast<int32_t>(q0);
        r.q_plane = groups.plane[g] + static_cast<int64_t>(local) * (QT / 128);
        r.p0 = static_cast<int64_t>(pt) * PT;
        r.p_row = static_cast<int32_t>(g * p.P + r.p0);
        r.p_plane = static_cast<int64_t>(g) * p.p_planes + pt * (PT / 128);
    } else {
        constexpr int kBand = 8;
        const int band = t / (kBand * p.p_tiles);
        const int in = t - band * kBand * p.p_tiles;
        const int width = min(kBand, p.q_tiles - band * kBand);
        const int pt = in / width, qt = band * kBand + in - pt * width;
        const int64_t left = p.Q - static_cast<int64_t>(qt) * QT;
        r.valid = left < QT ? static_cast<int>(left) : QT;
        r.q_row = qt * QT;
        r.q_plane = static_cast<int64_t>(qt) * (QT / 128);
        r.p0 = static_cast<int64_t>(pt) * PT;
        r.p_row = static_cast<int32_t>(r.p0);
        r.p_plane = pt * (PT / 128);
    }
    return r;
}

template <bool F32>
__device__ __forceinline__ void store_out(void *out, int64_t at, uint32_t bits)
{
    if constexpr (F32)
        static_cast<float *>(out)[at] = __uint_as_float(bits);
    else
        static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(__uint_as_float(bits));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(lo))) | (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(hi))) << 16);
}

// ---- epilogue --------------------------------------------------------------------------------------------
// A warp holds 32 output columns (its lanes) of 32 rows (registers).  Where output rows are whole 16-byte vectors
// the four warps transpose through shared memory and write 32 rows of 128 columns in 16-byte pieces: a warp then
// writes two 256-byte (fp32: one 512-byte) row pieces per instruction instead of 32 elements of one row, which made the
// epilogue the bound (13 us per 256 x 256 tile, twice the time of its MMAs at K = 4096).

constexpr int kEpiRows = 32;
template <bool F32>
constexpr int kEpiBytes = 2 * kEpiRows * kGemmRows * (F32 ? 4 : 2);  // two buffers

__device__ __forceinline__ void epilogue_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
// Whether all 128 epilogue threads say so.
__device__ __forceinline__ bool epilogue_all(bool ok)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(static_cast<uint32_t>(ok))
                 : "memory");
    return r != 0;
}

// Rows q0 .. q0 + 31 (of which `rows` are written) of 128 columns from col0; quarter: the warp's 32 lanes.  ADDS (fp32, vectors):
// where `add`, to what the same call has stored there before, each thread its own elements.
template <bool F32, bool ADDS = false>
__device__ __forceinline__ void store_chunk(const GemmParams &p, const uint32_t (&v)[32], unsigned char *buffer, int quarter, int lane,
                                            int64_t row0, int rows, int64_t col0, bool add = false)
{
    constexpr int kSize = F32 ? 4 : 2;
    if (!p.vec_out) {
        const int64_t col = col0 + quarter * 32 + lane;
        if (col < p.P) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j < rows)
                    store_out<F32>(p.out, (row0 + j) * p.ldo + col, v[j]);
        }
        return;
    }
    constexpr int kRowBytes = kGemmRows * kSize;
    unsigned char *dst = buffer + (quarter * 32 + lane) * kSize;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        if constexpr (F32)
            *reinterpret_cast<uint32_t *>(dst + j * kRowBytes) = v[j];
        else
            *reinterpret_cast<__nv_bfloat16 *>(dst + j * kRowBytes) = __float2bfloat16_rn(__uint_as_float(v[j]));
    }
    epilogue_sync();
    constexpr int kVecs = kRowBytes / 16, kPerPass = 128 / kVecs;
    const int tid = quarter * 32 + lane;
    const int vec = tid % kVecs, r0 = tid / kVecs;
    const bool live = col0 + vec * (16 / kSize) < p.P;
    unsigned char *out = static_cast<unsigned char *>(p.out) + ((row0 + r0) * p.ldo + col0) * kSize + vec * 16;
#pragma unroll
    for (int i = 0; i < kEpiRows / kPerPass; ++i) {
        uint4 q = *reinterpret_cast<const uint4 *>(buffer + (r0 + i * kPerPass) * kRowBytes + vec * 16);
        if (live && r0 + i * kPerPass < rows) {
            uint4 *to = reinterpret_cast<uint4 *>(out + static_cast<int64_t>(i) * kPerPass * p.ldo * kSize);
            if (ADDS && add) {
                const float4 b = *reinterpret_cast<const float4 *>(to), s = *reinterpret_cast<const float4 *>(&q);
                *reinterpret_cast<float4 *>(to) = make_float4(b.x + s.x, b.y + s.y, b.z + s.z, b.w + s.w);
            } else {
                *to = q;
            }
        }
    }
}

// The same where PARTS consecutive rows are parts of one: their sums, the smallest (the last) first.  A warp writes 32
// neighbouring columns of each of the 32 / PARTS rows.
template <bool F32, int PARTS>
__device__ __forceinline__ void store_parts(const GemmParams &p, const uint32_t (&v)[32], int quarter, int lane, int64_t row0, int rows, int64_t col0)
{
    const int64_t col = col0 + quarter * 32 + lane;
#pragma unroll
    for (int t = 0; t < 32 / PARTS; ++t) {
        float sum = __uint_as_float(v[PARTS * t + PARTS - 1]);
#pragma unroll
        for (int j = PARTS - 2; j >= 0; --j)
            sum += __uint_as_float(v[PARTS * t + j]);
        if (col < p.P && PARTS * t < rows)
            store_out<F32>(p.out, (row0 / PARTS + t) * p.ldo + col, __float_as_uint(sum));
    }
}

// The 128 epilogue threads of every CTA: zeros to the output's rows from `begin` on, which belong to no expert (ldo = P).
template <bool F32, int PARTS = 1>
__device__ __forceinline__ void clear_rows_from(const GemmParams &p, int64_t begin, int thread)
{
    constexpr int kVec = F32 ? 4 : 8;
    const int64_t first = begin / PARTS * p.P, last = p.Q / PARTS * p.P;
    const int64_t at = blockIdx.x * int64_t{128} + thread, step = gridDim.x * int64_t{128};
    if (p.vec_out) {
        for (int64_t i = first / kVec + at; i < last / kVec; i += step)
            static_cast<uint4 *>(p.out)[i] = make_uint4(0, 0, 0, 0);
    } else {
        for (int64_t i = first + at; i < last; i += step)
            store_out<F32>(p.out, i, 0u);
    }
}

// PARTS: consecutive rows of Q that are parts of one row of the output (mxfp4_parts.cuh); offsets then count output rows.
template <bool F32, int PARTS>
__global__ void __launch_bounds__(kGemmThreads, 1)
    mxfp4_group_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map, const GemmParams p)
{
    extern __shared__ unsigned char gemm_smem[];
    __shared__ GroupTable<true> groups;
    __shared__ uint64_t full[kGroupStages], empty[kGroupStages], acc_full[2], acc_empty[2], drain;
    __shared__ uint32_t tmem_slot;

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // warp-uniform for the compiler too
    const uint32_t base = (smem_u32(gemm_smem) + 1023u) & ~1023u;
    if (tid == 0) {
        prefetch_tensormap(&p_map);
        prefetch_tensormap(&q_map);
        for (int s = 0; s < kGroupStages; ++s) {
            mbar_init(smem_u32(&full[s]), 2);  // codes, scales
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), 4);
        }
        mbar_init(smem_u32(&drain), 1);
        fence_mbar_init();
    }
    if (warp == 2)
        tmem_alloc(smem_u32(&tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    if constexpr (PARTS == 1)
        pdl_wait_and_release();

    const int row_tiles = group_setup<kGemmThreads, kGemmRows, PARTS>(groups, p.offsets, p.num_groups, p.Q);
    const int num_tiles = row_tiles < 0 ? 0 : row_tiles * p.p_tiles;
    if (blockIdx.x == 0 && tid == 0 && p.err_flag != nullptr && (row_tiles < 0 || groups.offset[p.num_groups] < p.Q))
        atomicOr(p.err_flag, 1);
    auto give_up = [&]() { atomicOr(p.fault, 1u); };

    // stage of the ring and the phase parity of its barriers, for a role's next iteration
    int slot = 0;
    uint32_t phase = 0;
    auto advance = [&]() {
        if (++slot == kGroupStages) {
            slot = 0;
            phase ^= 1;
        }
    };
    const uint32_t full0 = smem_u32(&full[0]), empty0 = smem_u32(&empty[0]);
    // With parts, the kernel before on the stream writes Q alone, and began after all before it had ended: the weights of the
    // first stages are loaded while it runs.
    int early = 0;
    if constexpr (PARTS > 1) {
        if (static_cast<int>(blockIdx.x) < num_tiles && (warp == 0 || warp == 3)) {
            const GemmTile c = gemm_tile<kGemmRows, kGemmRows, true>(blockIdx.x, p, groups);
            const int boxes = (c.valid + p.q_box - 1) / p.q_box;
            early = min(kGroupStages, p.k_iters);
            for (int k = 0; k < early; ++k) {
                if (elect_one()) {
                    const uint32_t bar = full0 + 8 * k, dp = base + k * kGroupStage;
                    if (warp == 0) {
                        mbar_arrive_expect_tx(bar, kGroupBytes + boxes * p.q_box * 128);
                        tma_load_2d_shared(dp, &p_map, bar, k * 128, c.p_row);
                    } else {
                        const uint32_t sb = 512u * min(2, p.kc - 2 * k);
                        mbar_arrive_expect_tx(bar, 2 * sb);
                        bulk_load(dp + 2 * kGroupBytes, p.p_scale + c.p_plane * p.kc * 512 + int64_t{k} * 1024, sb, bar);
                    }
                }
                __syncwarp();
            }
        }
        pdl_wait_and_release();
    }

    if (warp == 0 || warp == 3) {
        // ---- producers: codes (warp 0), scales (warp 3) ----
        bool ok = true;
        int issued = 0;
        for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
            const GemmTile c = gemm_tile<kGemmRows, kGemmRows, true>(t, p, groups);
            const int boxes = (c.valid + p.q_box - 1) / p.q_box;
            const uint32_t code_bytes = kGroupBytes + boxes * p.q_box * 128;
            const uint8_t *ps = p.p_scale + c.p_plane * p.kc * 512, *qs = p.q_scale + c.q_plane * p.kc * 512;
            for (int k = 0; k < p.k_iters; ++k) {
                // a fresh barrier's phase -1 counts as complete: the first round waits for nothing
                ok = mbar_wait_cycles(empty0 + 8 * slot, phase ^ 1, kGemmWait);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = full0 + 8 * slot, dp = base + slot * kGroupStage;
                const bool started = PARTS > 1 && issued < early;  // its weights are on their way
                if (elect_one()) {
                    if (warp == 0) {
                        if (!started) {
                            mbar_arrive_expect_tx(bar, code_bytes);
                            tma_load_2d_shared(dp, &p_map, bar, k * 128, c.p_row);
                        }
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d_shared(dp + kGroupBytes + b * p.q_box * 128, &q_map, bar, k * 128, c.q_row + b * p.q_box);
                    } else {
                        const uint32_t sb = 512u * min(2, p.kc - 2 * k), ds = dp + kGroupBytes + kGroupBytes;
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
        }
        if (!ok) {
            if (lane == 0)
                give_up();
            for (int j = 0; j < kGroupStages && j < issued; ++j) {  // copies in flight, the newest first
                if (--slot < 0) {
                    slot = kGroupStages - 1;
                    phase ^= 1;
                }
                mbar_wait_cycles(full0 + 8 * slot, phase, kGemmDrain);
            }
        }
    } else if (warp == 1) {
        // ---- MMA ----
        int n_tile = 0;
        bool ok = true;
        const uint64_t p_desc = desc_sw128(base), q_desc = desc_sw128(base + kGroupBytes);
        const uint64_t s_desc = desc_scales(base + kGroupBytes + kGroupBytes);
        for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x, ++n_tile) {
            const GemmTile c = gemm_tile<kGemmRows, kGemmRows, true>(t, p, groups);
            const int n = (c.valid + 15) & ~15;
            const int buf = n_tile & 1;
            const uint32_t d = tmem + buf * kGemmRows, sf = tmem + kGroupScaleCol;
            const uint32_t idesc0 = mxf4_idesc(kGemmRows, n, 0), idesc1 = mxf4_idesc(kGemmRows, n, 1);
            if (n_tile >= 2)
                ok = mbar_wait_cycles(smem_u32(&acc_empty[buf]), ((n_tile >> 1) - 1) & 1, kGemmWait);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            for (int k = 0; k < p.k_iters; ++k) {
                ok = mbar_wait_cycles(full0 + 8 * slot, phase, kGemmWait);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t step = slot * (kGroupStage >> 4);  // descriptors count 16-byte units
                    const uint64_t pd = p_desc + step, qd = q_desc + step, sd = s_desc + step;
                    const int left = p.k64 - 4 * k;  // MMA steps from here on
#pragma unroll
                    for (int ch = 0; ch < 2; ++ch) {
                        if (left <= 2 * ch)
                            break;
                        // each half of a stage has its own TMEM columns for its scales; copies and MMAs run in issue order
                        const uint32_t sp = sf + ch * (8), sq = sp + 4;
                        tc_copy_scales(sp, sd + ch * 32);
                        tc_copy_scales(sq, sd + (1024 + ch * 512) / 16);
                        tc_mma_mxf4(d, pd + ch * 4, qd + ch * 4, idesc0, sp, sq, k > 0 || ch > 0);
                        if (left > 2 * ch + 1)
                            tc_mma_mxf4(d, pd + ch * 4 + 2, qd + ch * 4 + 2, idesc1, sp, sq, true);
                    }
                    tc_commit(empty0 + 8 * slot);
                    if (k == p.k_iters - 1)
                        tc_commit(smem_u32(&acc_full[buf]));
                }
                __syncwarp();
                advance();
            }
        }
        if (!ok) {
            if (elect_one()) {
                give_up();
                tc_commit(smem_u32(&drain));
            }
            __syncwarp();
            mbar_wait_cycles(smem_u32(&drain), 0, kGemmDrain);
        }
    } else if (warp >= 4) {
        // ---- epilogue ----
        const int quarter = warp & 3;
        unsigned char *stage_out = gemm_smem + (base - smem_u32(gemm_smem)) + kGroupStages * kGroupStage;
        int n_tile = 0, chunk = 0;
        if (row_tiles >= 0)
            clear_rows_from<F32, PARTS>(p, groups.offset[p.num_groups], quarter * 32 + lane);
        for (int t = blockIdx.x; t < num_tiles; t += gridDim.x, ++n_tile) {
            const GemmTile c = gemm_tile<kGemmRows, kGemmRows, true>(t, p, groups);
            const int buf = n_tile & 1;
            if (!epilogue_all(mbar_wait_cycles(smem_u32(&acc_full[buf]), (n_tile >> 1) & 1, kGemmWait))) {
                if (lane == 0)
                    give_up();
                break;
            }
            tc_fence_after();
            for (int q = 0; q < c.valid; q += 32) {
                uint32_t v[32];
                tmem_load32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * kGemmRows + q, v);
                if constexpr (PARTS > 1)
                    store_parts<F32, PARTS>(p, v, quarter, lane, c.q_row + q, c.valid - q, c.p0);
                else
                    store_chunk<F32>(p, v, stage_out + (chunk++ & 1) * (kEpiBytes<F32> / 2), quarter, lane, c.q_row + q, c.valid - q, c.p0);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&acc_empty[buf]));
        }
    }
    __syncthreads();
    if (warp == 2)
        tmem_dealloc(tmem, 512);
}

}  // namespace mxfp8
