// Experts' products in MXFP8 (sm_103a) by pairs of CTAs: out[q, p] = sum_k Q[q, k] * P[p, k] in tiles of 256 x 256.
//
//   forward           Q = x's rows, P = W's rows           summed over K, both operands K-major
//   input gradient    Q = dy's rows, P = W's columns       summed over N: P's codes lie [N, K], MN-major
//   weight gradient   P = dy's columns, Q = x's columns    summed over the expert's rows: both MN-major; out[p, q]
//
// The cast leaves the columns' codes untransposed ([rows, columns], blocks of 32 rows), so the gradients read them as
// MN-major operands: a TMA box of 128 summed rows x 128 bytes in the 128-byte swizzle is one operand atom wide, and a step
// of 32 summed elements is 32 of its rows.  No transposed copy exists.
//
// The loop is that of mxfp4_pair.cuh: 128 bytes of codes per operand row and stage, here 128 elements in four MMA steps
// of 32 (kind::mxf8f6f4, one E8M0 scale per step and row); the accumulators share 32 TMEM columns as there.  Tiles of 192
// columns, whose two accumulators share nothing, were slower throughout (8192x8192x8192 312 -> 356 us): operand loads.
//
// A weight gradient's last stage may hold rows of the next expert.  Steps past the expert's last 32 rows are not issued;
// where the rows are no multiple of 32 each CTA's warp 2 zeroes the rest of the last step in shared memory before the MMA warp
// sees the stage: copies from before the codes' first row, which read zeros, once its own barrier says that the codes have
// landed.  Like the codes they signal the first CTA's barrier, which expects them in the codes' place, so that nothing but
// copies orders them before the MMAs that the first CTA issues for both.  (Generic stores need a release and an acquire at
// cluster scope for that: 64 experts of 1024 rows on average, fp32 out, 1130 us against 970.)
//
// The tensor core truncates its fp32 sums (one rounds them): an error toward zero that grows with their length, and faster where
// tokens differ in scale.  To fp32 a sum is made in pieces of kP8Piece stages, each in a fresh accumulator, added in order: of
// 2048 rows for the weight gradient, in the epilogue's registers (an epilogue warp keeps its columns through a tile), of 8192
// elements for the other two, in the output.  Norm-wise error against 64 bits of a weight gradient of 2048, 8192 and 65536
// rows: normal values 0.7e-7, 0.9e-7, 1.3e-7 (in one piece 0.7e-7, 3.0e-7, 45e-7; a plain fp32 product 0.4e-7, 0.6e-7, 1.2e-7); rows
// scaled by exp of a normal value 3.1e-7, 3.5e-7, 4.2e-7 (in one piece 3.1e-7, 20e-7, 244e-7).  8192x8192x8192 to fp32 333 -> 359 us, 8
// experts of 8192 rows 538 -> 576, of up to 2048 rows as before; pieces added in the output took 548 and 970.  To bf16 the
// truncation is far below the rounding, and a sum is one piece.
//
// Measured: 8192x8192x8192 312 us (3.5 PFLOP/s; the bf16 rate measured with cuBLAS twice over is 3.8), 64 experts of 1024 rows on
// average, 7168 -> 2048: forward 598 us, input gradient 632, weight gradient 970 to fp32 (912 where every expert has 1024; the 3.76 GB
// that it writes take 553 at the copy rate) and 755 to bf16 (697); two rows per expert 153, 146, 607 and 354.  Many rows: bound by the
// MMAs under the power limit (tensor pipe active 73% of the forward's cycles), the ragged last tile of each expert and, for the
// weight gradient, most likely the path from the SMs to L2 (requests in close to 60% of its cycles, DRAM 4.1 TB/s, tensor pipe 41%):
// a stage's loads take 3600 to 4200 cycles while tiles are stored.  Few: the weights' bytes (6.3 TB/s), or the gradient's.
#pragma once

#include "mxfp4_gemm.cuh"

namespace mxfp8 {

enum { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

constexpr int kP8Tile = 256;
constexpr int kP8Stages = 5;
constexpr int kP8Codes = 128 * 128;           // bytes of either operand in one CTA and stage
constexpr int kP8Stage = 2 * kP8Codes;
constexpr int kP8Scales = 3 * 512;            // P's tile of this CTA, Q's two tiles
constexpr int kP8Epi = (kP8Stages * (kP8Stage + kP8Scales) + 1023) / 1024 * 1024;  // the epilogue's buffers from here on
constexpr int kP8Smem = kP8Epi + 1024;
constexpr int kP8Acc1 = 224, kP8ScaleCol = 480;  // TMEM columns, as in mxfp4_pair.cuh

// Stages of a piece of a sum to fp32.
template <int MODE>
constexpr int kP8Piece = MODE == kWeightGrad ? 16 : 64;
template <int MODE, bool F32>
__device__ __forceinline__ int sum_pieces(int k_iters)
{
    return F32 && k_iters > kP8Piece<MODE> ? (k_iters + kP8Piece<MODE> - 1) / kP8Piece<MODE> : 1;
}

// The boxes of zeros that cover `rows` (1 to 31) rows: of 8 rows, the last one back over rows that are zero already, or of one.
constexpr int kZeroRows = 8;
struct ZeroBoxes {
    int rows, count;  // of a box; boxes
};
__device__ __forceinline__ ZeroBoxes zero_boxes(int rows)
{
    return rows >= kZeroRows ? ZeroBoxes{kZeroRows, (rows + kZeroRows - 1) / kZeroRows} : ZeroBoxes{1, rows};
}

// A weight gradient's tile has few stages and many bytes to write: eight epilogue warps, with a buffer of 32 rows x 128
// bytes each (four warps with two each, 64 experts of 2048 x 7168, bf16 out: two rows each 352 against 527 us, 1024 rows
// each 719 against 763).
template <int MODE>
constexpr int kP8Threads = MODE == kWeightGrad ? 384 : kGemmThreads;
template <int MODE, bool F32>
constexpr int kP8Epilogue = MODE == kWeightGrad ? 8 * 4096 : kEpiBytes<F32>;

struct Product8Params : GemmParams {
    uint32_t formats;      // operand format bits of the instruction descriptor
    int64_t sum;           // summed elements; weight gradient: rows of all experts
    int64_t p_tile_rows;   // tile rows that the ragged planes hold (weight gradient: tiles)
    int64_t q_tile_rows;
    int p_ct, q_ct;        // weight gradient: 128-column tiles of either operand's planes
};

struct Tile8 {
    int32_t p_at, q_at, row;   // P's first row (K-major) or column; Q's; weight gradient: the expert's first row
    int32_t group;
    int64_t p_tile, q_tile;    // scale tile rows; weight gradient: linear tiles
    int64_t out_row;           // of [total_rows, P]
    int valid, k_iters, steps, tail;  // rows of Q; stages; MMA steps in all; rows of the last step (0: whole)
    int kt;            // weight gradient: scale tiles along the rows
};

template <int MODE>
__device__ __forceinline__ Tile8 tile8(int t, const Product8Params &p, const GroupTable<true> &groups)
{
    Tile8 r;
    if constexpr (MODE == kWeightGrad) {
        const int per = p.p_tiles * p.q_tiles;
        const int g = t / per, in = t - g * per, qt = in / p.p_tiles, pt = in - qt * p.p_tiles;
        const int64_t rows = groups.offset[g + 1] - groups.offset[g];
        r.group = g;
        r.row = static_cast<int32_t>(groups.offset[g]);
        r.p_at = pt * kP8Tile;
        r.q_at = qt * kP8Tile;
        r.kt = groups.plane[g + 1] - groups.plane[g];
        r.p_tile = static_cast<int64_t>(groups.plane[g]) * p.p_ct + static_cast<int64_t>(2 * pt) * r.kt;
        r.q_tile = static_cast<int64_t>(groups.plane[g]) * p.q_ct + static_cast<int64_t>(r.q_at / 128) * r.kt;
        r.out_row = 0;
        const int64_t left = p.Q - r.q_at;
        r.valid = left < kP8Tile ? static_cast<int>(left) : kP8Tile;
        r.k_iters = r.kt;
        r.steps = static_cast<int>((rows + 31) / 32);
        r.tail = static_cast<int>(rows & 31);
    } else {
        const int rt = t / p.p_tiles, pt = t - rt * p.p_tiles;
        const int g = groups.find(rt, p.num_groups);
        const int local = rt - groups.tile[g];
        const int64_t q0 = groups.offset[g] + static_cast<int64_t>(local) * kP8Tile;
        const int64_t left = groups.offset[g + 1] - q0;
        r.group = g;
        r.row = 0;
        r.p_at = pt * kP8Tile;
        r.q_at = static_cast<int32_t>(q0);
        r.kt = 0;
        r.p_tile = static_cast<int64_t>(g) * p.p_planes + 2 * pt;
        r.q_tile = groups.plane[g] + static_cast<int64_t>(local) * (kP8Tile / 128);
        r.out_row = q0;
        r.valid = left < kP8Tile ? static_cast<int>(left) : kP8Tile;
        r.k_iters = p.k_iters;
        r.steps = static_cast<int>((p.sum + 31) / 32);
        r.tail = 0;
    }
    return r;
}

// 3-D tiled copy into this CTA's shared memory that signals a barrier of either CTA of its pair.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, uint32_t mapped_bar, int32_t x, int32_t y, int32_t z)
{
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(mapped_bar)
                 : "memory");
}

// Operand whose summed dimension lies across rows of 128 bytes (MN-major, 128-byte swizzle): groups of 8 summed rows 1024
// bytes apart; one atom of 128 elements wide, so the other stride is not used (set to the same, within the stage).
__device__ __forceinline__ uint64_t desc_mn128(uint32_t smem)
{
    return static_cast<uint64_t>((smem & 0x3FFFF) >> 4) | (uint64_t{1024 >> 4} << 16) | (uint64_t{1024 >> 4} << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

// Tiled store of one box from this CTA's shared memory; bulk_store_wait<N>: all but the thread's last N have read theirs.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int32_t x, int32_t y, int32_t z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n\tcp.async.bulk.commit_group;" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void bulk_store_wait()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Instruction descriptor of kind::mxf8f6f4 with E8M0 scales; formats: operand formats at bits 7 and 10, transposes at 15
// and 16; step: which of a TMEM column's four scales the 32 elements of this step use.
__device__ __forceinline__ uint32_t mxf8_idesc(uint32_t formats, int m, int n, int step)
{
    return formats | (static_cast<uint32_t>(step) << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(m >> 7) << 27) | (static_cast<uint32_t>(step) << 29);
}

__device__ __forceinline__ void tc_mma_mxf8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, bool accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(static_cast<uint32_t>(accumulate))
                 : "memory");
}

template <int MODE, bool F32>
__global__ void __launch_bounds__(kP8Threads<MODE>, 1)
    mxfp8_pair_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap q_part_map, const __grid_constant__ CUtensorMap ps_map,
                      const __grid_constant__ CUtensorMap qs_map, const __grid_constant__ CUtensorMap out_map,
                      const __grid_constant__ CUtensorMap zeros_map, const __grid_constant__ CUtensorMap zero_row_map, const Product8Params p)
{
    constexpr bool kTails = MODE == kWeightGrad;
    constexpr bool kPMn = MODE != kForward, kQMn = MODE == kWeightGrad;
    extern __shared__ unsigned char gemm_smem[];
    __shared__ GroupTable<true> groups;
    __shared__ uint64_t full[kP8Stages], empty[kP8Stages], landed[kP8Stages], acc_full[2], acc_empty, drain;
    __shared__ uint32_t tmem_slot;

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const uint32_t rank = cluster_rank();
    const uint32_t base = (smem_u32(gemm_smem) + 1023u) & ~1023u;
    const uint32_t scales = base + kP8Stages * kP8Stage;
    if (tid == 0) {
        prefetch_tensormap(&p_map);
        prefetch_tensormap(&q_map);
        prefetch_tensormap(&q_part_map);
        prefetch_tensormap(&ps_map);
        prefetch_tensormap(&qs_map);
        prefetch_tensormap(&out_map);
        if (kTails) {
            prefetch_tensormap(&zeros_map);
            prefetch_tensormap(&zero_row_map);
        }
        for (int s = 0; s < kP8Stages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
            mbar_init(smem_u32(&landed[s]), 1);
        }
        mbar_init(smem_u32(&acc_full[0]), 1);
        mbar_init(smem_u32(&acc_full[1]), 1);
        mbar_init(smem_u32(&acc_empty), kTails ? 16 : 8);  // the epilogue warps of both CTAs
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

    int rt = group_setup<kP8Threads<MODE>, kP8Tile>(groups, p.offsets, p.num_groups, MODE == kWeightGrad ? p.sum : p.Q);
    const int64_t total = MODE == kWeightGrad ? p.sum : p.Q;
    if (rt >= 0) {  // offsets that need larger planes than there are
        const int64_t tiles = groups.plane[p.num_groups];
        if (MODE == kWeightGrad ? tiles * p.q_ct > p.q_tile_rows || tiles * p.p_ct > p.p_tile_rows : tiles > p.q_tile_rows)
            rt = -1;
    }
    const int num_tiles = rt < 0 ? 0 : MODE == kWeightGrad ? p.num_groups * p.p_tiles * p.q_tiles : rt * p.p_tiles;
    const int64_t no_expert = rt < 0 ? total : groups.offset[p.num_groups];  // the first row of no expert
    if (blockIdx.x == 0 && tid == 0 && p.err_flag != nullptr && (rt < 0 || no_expert < total))
        atomicOr(p.err_flag, 1);
    // the pair's n-th tile: rounds of one tile per pair, every other one backwards (as in mxfp4_pair.cuh)
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    auto tile_of = [&](int n) { return n * pairs + (n & 1 ? pairs - 1 - pair : pair); };
    const uint32_t full0 = smem_u32(&full[0]), empty0 = smem_u32(&empty[0]), landed0 = smem_u32(&landed[0]);
    int slot = 0;
    uint32_t phase = 0;
    auto advance = [&]() {
        if (++slot == kP8Stages) {
            slot = 0;
            phase ^= 1;
        }
    };

    // the next piece of a tile's sum, or the next tile
    auto next_piece = [&](const Tile8 &c, int &piece, int &n_tile) {
        if (++piece == sum_pieces<MODE, F32>(c.k_iters)) {
            piece = 0;
            ++n_tile;
        }
    };

    if (warp == 0 || warp == 3) {
        // ---- producers of this CTA's operands: codes (warp 0), scales (warp 3); they signal the first CTA's barriers ----
        const uint32_t lead_full = map_to_rank(full0, 0), own_landed = map_to_rank(landed0, rank);
        bool ok = true;
        int issued = 0;
        for (int n = 0, t; (t = tile_of(n)) < num_tiles && ok; ++n) {
            const Tile8 c = tile8<MODE>(t, p, groups);
            const int half = ((c.valid + 31) & ~31) / 2;
            const int boxes = kQMn || half > kP8Tile / 2 - 32 ? 0 : (half + 31) / 32;  // a partial tile's rows of Q in boxes of 32 (0: whole)
            const uint32_t code_bytes = kP8Codes + (kQMn ? kP8Codes : boxes ? boxes * 32 * 128 : kP8Tile / 2 * 128);
            for (int k = 0; k < c.k_iters; ++k) {
                ok = mbar_wait_cycles(empty0 + 8 * slot, phase ^ 1, kGemmWait);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    const bool zeroed = kTails && c.tail != 0 && k == c.k_iters - 1;
                    const uint32_t dp = base + slot * kP8Stage;
                    if (warp == 0) {
                        if (rank == 0) {
                            uint32_t bytes = code_bytes;
                            if (zeroed) {  // the rows behind the expert's last, of both operands, once the codes have landed
                                const ZeroBoxes z = zero_boxes(32 - c.tail);
                                bytes = 2 * z.count * z.rows * 128;
                            }
                            mbar_arrive_expect_tx(full0 + 8 * slot, 2 * (kP8Scales + bytes));
                        }
                        if (zeroed)
                            mbar_arrive_expect_tx(landed0 + 8 * slot, code_bytes);
                        const uint32_t bar = (zeroed ? own_landed : lead_full) + 8 * slot;
                        const int p_at = c.p_at + static_cast<int>(rank) * 128, q_at = c.q_at + static_cast<int>(rank) * half;
                        if constexpr (MODE == kForward)
                            tma_load_3d_pair(dp, &p_map, bar, k * 128, p_at, c.group);
                        else if constexpr (MODE == kInputGrad)
                            tma_load_3d_pair(dp, &p_map, bar, p_at, k * 128, c.group);
                        else
                            tma_load_2d_pair(dp, &p_map, bar, p_at, c.row + k * 128);
                        if constexpr (kQMn) {
                            tma_load_2d_pair(dp + kP8Codes, &q_map, bar, q_at, c.row + k * 128);
                        } else {
                            if (boxes == 0)
                                tma_load_2d_pair(dp + kP8Codes, &q_map, bar, k * 128, q_at);
                            for (int b = 0; b < boxes; ++b)
                                tma_load_2d_pair(dp + kP8Codes + b * 32 * 128, &q_part_map, bar, k * 128, q_at + 32 * b);
                        }
                    } else {
                        const uint32_t bar = lead_full + 8 * slot, ds = scales + slot * kP8Scales;
                        if constexpr (MODE == kWeightGrad) {
                            tma_load_2d_pair(ds, &ps_map, bar, 0, static_cast<int>(c.p_tile + static_cast<int64_t>(rank) * c.kt + k));
                            tma_load_2d_pair(ds + 512, &qs_map, bar, 0, static_cast<int>(c.q_tile + k));
                            tma_load_2d_pair(ds + 1024, &qs_map, bar, 0, static_cast<int>(c.q_tile + c.kt + k));
                        } else {
                            tma_load_2d_pair(ds, &ps_map, bar, k * 128, static_cast<int>(c.p_tile) + static_cast<int>(rank));
                            tma_load_2d_pair(ds + 512, &qs_map, bar, k * 128, static_cast<int>(c.q_tile));
                        }
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
            for (int j = 0; j < kP8Stages && j < issued; ++j) {  // copies in flight, the newest first
                if (--slot < 0) {
                    slot = kP8Stages - 1;
                    phase ^= 1;
                }
                mbar_wait_cycles(full0 + 8 * slot, phase, kGemmDrain);
            }
        }
    } else if (kTails && warp == 2) {
        // ---- zeros behind an expert's last row, in this CTA's shared memory ----
        const uint32_t lead_full = map_to_rank(full0, 0);
        uint32_t phases = 0;
        for (int n = 0, t; (t = tile_of(n)) < num_tiles; ++n) {
            const Tile8 c = tile8<MODE>(t, p, groups);
            if (c.tail != 0) {
                const int s = (slot + c.k_iters - 1) % kP8Stages;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait_cycles(landed0 + 8 * s, (phases >> s) & 1, kGemmWait))) {
                    if (lane == 0)
                        atomicOr(p.fault, 1u);
                    break;
                }
                phases ^= 1u << s;
                const int rows = 32 - c.tail, end = (c.steps - 1) % 4 * 32 + 32;  // the last step's, within the stage
                const ZeroBoxes z = zero_boxes(rows);
                if ((lane & 15) < z.count) {  // lanes from 0 on: P's boxes, from 16 on: Q's.  Whole rows: the swizzle stays inside
                    const int at = min(end - rows + (lane & 15) * z.rows, end - z.rows);
                    const uint32_t dst = base + s * kP8Stage + (lane >> 4) * kP8Codes + at * 128;
                    tma_load_2d_pair(dst, z.rows == 1 ? &zero_row_map : &zeros_map, lead_full + 8 * s, 0, -z.rows);
                }
                __syncwarp();
            }
            slot = (slot + c.k_iters) % kP8Stages;
        }
    } else if (warp == 1 && rank == 0) {
        // ---- MMA for both CTAs ----
        bool ok = true;
        constexpr uint32_t kPStep = kPMn ? 4096 / 16 : 32 / 16, kQStep = kQMn ? 4096 / 16 : 32 / 16;
        const uint64_t p_desc = kPMn ? desc_mn128(base) : desc_sw128(base);
        const uint64_t q_desc = kQMn ? desc_mn128(base + kP8Codes) : desc_sw128(base + kP8Codes);
        const uint64_t s_desc = desc_scales(scales);
        const uint32_t formats = p.formats | (kPMn ? 1u << 15 : 0u) | (kQMn ? 1u << 16 : 0u);
        int piece = 0, k0 = 0;  // of the tile's sum, and its first stage
        for (int n_tile = 0, acc = 0, t; (t = tile_of(n_tile)) < num_tiles && ok; ++acc) {  // acc: accumulators so far
            const Tile8 c = tile8<MODE>(t, p, groups);
            const int n = (c.valid + 31) & ~31;  // halves of whole 16-row groups
            const int buf = acc & 1;
            const uint32_t d = tmem + buf * kP8Acc1;
            if (acc >= 1)  // the columns shared with the accumulator before are read, and all of the one before that
                ok = mbar_wait_cycles(smem_u32(&acc_empty), (acc - 1) & 1, kGemmWait);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int k1 = sum_pieces<MODE, F32>(c.k_iters) > 1 ? min(c.k_iters, k0 + kP8Piece<MODE>) : c.k_iters;
            for (int k = k0; k < k1; ++k) {
                ok = mbar_wait_cycles(full0 + 8 * slot, phase, kGemmWait);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t pd = p_desc + slot * (kP8Stage >> 4), qd = q_desc + slot * (kP8Stage >> 4), sd = s_desc + slot * (kP8Scales >> 4);
                    const uint32_t sp = tmem + kP8ScaleCol + (k & 1) * 12, sq = sp + 4;
                    const int left = c.steps - 4 * k;
                    tc_copy_scales_pair(sp, sd);
                    tc_copy_scales_pair(sq, sd + 512 / 16);
                    tc_copy_scales_pair(sq + 4, sd + 1024 / 16);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < left)
                            tc_mma_mxf8_pair(d, pd + j * kPStep, qd + j * kQStep, mxf8_idesc(formats, kP8Tile, n, j), sp, sq, k > k0 || j > 0);
                    tc_commit_pair(empty0 + 8 * slot);
                }
                __syncwarp();
                advance();
            }
            if (!ok)
                break;
            if (elect_one())
                tc_commit_pair(smem_u32(&acc_full[buf]));
            __syncwarp();
            next_piece(c, piece, n_tile);
            k0 = piece * kP8Piece<MODE>;
        }
        if (!ok) {
            if (elect_one()) {
                atomicOr(p.fault, 1u);
                tc_commit_pair(smem_u32(&drain));
            }
            __syncwarp();
            mbar_wait_cycles(smem_u32(&drain), 0, kGemmDrain);
        }
    } else if (kTails && warp >= 4) {
        // ---- epilogue of this CTA's 128 rows of an expert's gradient: a warp has 32 rows, a thread one ----
        constexpr int kCols = F32 ? 32 : 64, kChunks = kP8Tile / kCols;  // 128 bytes of a row
        // (two warps to 32 rows, a chunk of 128 bytes of each in turn)
        const int quarter = warp & 3, part = (warp - 4) >> 2;
        const uint32_t lead_empty = map_to_rank(smem_u32(&acc_empty), 0);
        unsigned char *buffer = gemm_smem + (base - smem_u32(gemm_smem)) + kP8Epi + (warp - 4) * 4096;
        float sum[F32 ? kChunks / 2 : 1][32];  // of the pieces before
        int piece = 0;
        for (int n_tile = 0, acc = 0, t; (t = tile_of(n_tile)) < num_tiles; ++acc) {
            const Tile8 c = tile8<MODE>(t, p, groups);
            const int buf = acc & 1;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_cycles(smem_u32(&acc_full[buf]), (acc >> 1) & 1, kGemmWait))) {
                if (lane == 0)
                    atomicOr(p.fault, 1u);
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * kP8Acc1;
            const int row = c.p_at + static_cast<int>(rank) * 128 + quarter * 32;
            // The columns that the accumulators share are the last chunk of buffer 0 and the first of buffer 1.  The warp that has them
            // frees them after its first chunk; the other one's share of the accumulator before is read.
            const bool shares = part == (buf ^ 1), more = piece + 1 < sum_pieces<MODE, F32>(c.k_iters);
            if (!shares) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_peer(lead_empty);
            }
#pragma unroll(F32 ? kChunks / 2 : 1)
            for (int i = 0; i < kChunks / 2; ++i) {
                const int q = kCols * (part == 0 ? 2 * i : (kChunks - 1 + 2 * i) % kChunks);
                const bool live = q < c.valid && row < p.P;
                uint32_t v[kCols];
                if (live) {
#pragma unroll
                    for (int h = 0; h < kCols / 32; ++h)
                        tmem_load32(d + q + 32 * h, *reinterpret_cast<uint32_t (*)[32]>(&v[32 * h]));
                }
                if (i == 0 && shares) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_peer(lead_empty);
                }
                if (!live)
                    continue;
                if constexpr (F32) {
                    if (piece > 0) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = __float_as_uint(sum[i][j] + __uint_as_float(v[j]));
                    }
                    if (more) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            sum[i][j] = __uint_as_float(v[j]);
                        continue;
                    }
                }
                if (lane == 0)
                    bulk_store_wait<0>();
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) {  // 16 bytes each, in the store's 128-byte swizzle
                    uint4 w;
                    if constexpr (F32)
                        w = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    else
                        w = make_uint4(pack_bf16x2(__uint_as_float(v[8 * j]), __uint_as_float(v[8 * j + 1])),
                                       pack_bf16x2(__uint_as_float(v[8 * j + 2]), __uint_as_float(v[8 * j + 3])),
                                       pack_bf16x2(__uint_as_float(v[8 * j + 4]), __uint_as_float(v[8 * j + 5])),
                                       pack_bf16x2(__uint_as_float(v[8 * j + 6]), __uint_as_float(v[8 * j + 7])));
                    if (c.k_iters == 0)  // an expert without rows
                        w = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(buffer + lane * 128 + ((j ^ (lane & 7)) * 16)) = w;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    tma_store_3d(&out_map, smem_u32(buffer), c.q_at + q, row, c.group);
            }
            next_piece(c, piece, n_tile);
        }
        if (lane == 0)
            bulk_store_wait<0>();
        __syncwarp();
    } else if (warp >= 4) {
        // ---- epilogue of this CTA's 128 columns of the output ----
        const int quarter = warp & 3;
        const uint32_t lead_empty = map_to_rank(smem_u32(&acc_empty), 0);
        unsigned char *stage_out = gemm_smem + (base - smem_u32(gemm_smem)) + kP8Epi;
        int chunk = 0;
        clear_rows_from<F32>(p, no_expert, quarter * 32 + lane);
        int piece = 0;
        for (int n_tile = 0, acc = 0, t; (t = tile_of(n_tile)) < num_tiles; ++acc) {
            const Tile8 c = tile8<MODE>(t, p, groups);
            const int buf = acc & 1;
            if (!epilogue_all(mbar_wait_cycles(smem_u32(&acc_full[buf]), (acc >> 1) & 1, kGemmWait))) {
                if (lane == 0)
                    atomicOr(p.fault, 1u);
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * kP8Acc1;
            const int start = buf == 0 ? kP8Acc1 : 0;  // the columns that the accumulators share first
            for (int i = 0; i < kP8Tile / 32; ++i) {
                const int q = (start + 32 * i) & (kP8Tile - 1);
                uint32_t v[32];
                if (q < c.valid)
                    tmem_load32(d + q, v);
                if (i == 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_peer(lead_empty);
                }
                if (q < c.valid)
                    store_chunk<F32, F32>(p, v, stage_out + (chunk++ & 1) * (kEpiBytes<F32> / 2), quarter, lane, c.out_row + q, c.valid - q,
                                          c.p_at + rank * 128, piece > 0);
            }
            next_piece(c, piece, n_tile);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its pair's MMAs, copies or arrivals may still reach it
    if (warp == 2)
        tmem_dealloc_pair(tmem, 512);
}

}  // namespace mxfp8
