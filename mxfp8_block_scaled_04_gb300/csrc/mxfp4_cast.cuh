// MXFP4 cast and its inverse (sm_103a); formulas and layouts in include/mxfp4.h.
//
// One pass over HBM.  CTAs take tiles of 128 rows x 256 bytes (128 BF16 or 64 fp32 columns) in turn, so that the
// tiles at work cover whole rows (a run of tiles per CTA instead measured 30% slower: it keeps ten times as many
// DRAM pages open), through a ring of shared-memory stages filled by 16-byte asynchronous copies, which serve gathered
// rows and ragged edges (zero fill) alike and keep the next tile in flight while one is cast.  Rowwise, a thread holds 32
// bytes of a row that it copied itself and a block is two (fp32: four) lanes; columnwise, a thread takes one word
// (two BF16 columns or one fp32) of 32 rows, so that the four lanes of a column write 64 consecutive bytes of the
// transposed codes.  HBM: 2 (or 4) bytes in and 17/32 byte out per element and direction; one way is bound by that
// (8192x28672 BF16: 97 us, 6.1 TB/s), both ways by the SM side as well (145 us, 5.0 TB/s; the issue slots are half
// used, and neither the conversions nor the tile order nor more stages change it).
//
// The scale exponent comes from the bits of amax (exact), x * 2^(127 - e) is exact wherever the rounding to
// E2M1 depends on it (powers of two, fp32 subnormals kept), so the codes are those of the definition.
#pragma once

#include <cstdint>
#include <type_traits>

#include "groups.cuh"
#include "ptx.cuh"

namespace mxfp8 {

constexpr int kCastThreads = 256;
constexpr int kCastTile = 128;

struct CastParams {
    const void *x;
    int64_t M, N, ldx;    // rows of the output, columns, input row pitch (elements)
    uint8_t *out_row, *scale_row, *out_col, *scale_col;
    const float *noop;
    int row_tiles, col_tiles;
    int64_t row_pitch, col_pitch;  // bytes of a row of codes, per direction
    // grouped
    const int32_t *rows;
    const int64_t *offsets;
    int *err_flag;
    int64_t T;            // rows of x
    int num_groups;
};

// The block's E8M0 byte from the fp32 bits of amax: ceil(log2(amax / 6)) + 127 with 6 = 1.5 * 2^2.
__device__ __forceinline__ int fp4_exponent(uint32_t amax)
{
    int e = static_cast<int>(amax >> 23) - 2 + ((amax & 0x7FFFFFu) > 0x400000u ? 1 : 0);
    e = e < 0 ? 0 : e;
    e = amax == 0 ? 127 : e;
    return amax >= 0x7F800000u ? 255 : e;
}

// 2^(127 - e); e = 255 (NaN block) gives 0, and the caller's codes are masked.
__device__ __forceinline__ float fp4_multiplier(int e) { return __uint_as_float(static_cast<uint32_t>(e == 255 ? 0 : 254 - e) << 23); }

// Eight fp32 -> eight E2M1 codes, v[0] in the low four bits.
__device__ __forceinline__ uint32_t cvt_fp4x8(const float *v)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight values times one multiplier (a splat pair) -> codes; the products as packed pairs.
__device__ __forceinline__ uint32_t cvt_fp4x8_scaled(const float *x, uint64_t mul)
{
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        f2_unpack(f2_mul(f2_pack(x[2 * j], x[2 * j + 1]), mul), v[2 * j], v[2 * j + 1]);
    return cvt_fp4x8(v);
}

// Two E2M1 codes (a byte) -> two fp32.
__device__ __forceinline__ void fp4x2_to_f32(uint32_t byte, float &lo, float &hi)
{
    uint32_t h;
    asm("{\n\t.reg .b8 b, z0, z1, z2;\n\tmov.b32 {b, z0, z1, z2}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(lo), "=f"(hi) : "r"(h));
}

__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The rows past the last group's, of no group: zero codes.  `rows` marks such a row with a negative index; any other
// one, and any at all without `rows`, is reported.
template <int THREADS>
__device__ __forceinline__ void clear_left_over(uint8_t *out, int64_t pitch, int64_t begin, int64_t end, const int32_t *rows, int *err_flag)
{
    if (begin >= end)
        return;
    const int64_t first = blockIdx.x * int64_t{THREADS} + threadIdx.x, step = gridDim.x * int64_t{THREADS};
    uint4 *to = reinterpret_cast<uint4 *>(out + begin * pitch);
    for (int64_t i = first; i < (end - begin) * pitch / 16; i += step)
        to[i] = make_uint4(0, 0, 0, 0);
    bool lost = rows == nullptr && first == 0;
    if (rows != nullptr)
        for (int64_t r = begin + first; r < end; r += step)
            lost |= rows[r] >= 0;
    if (lost && err_flag != nullptr)
        atomicOr(err_flag, 1);
}

// Stages of 128 rows of 64 words; each group of 32 rows is shifted by a quarter of the banks, so that a warp's
// reads of 8 words x 4 row blocks hit 32 banks.
constexpr int kCastWords = 64;
constexpr int kCastStages = 2;  // 3 measured 5% slower both ways, 3 CTAs per SM no faster
constexpr int kCastStage = (kCastTile * kCastWords + 3 * 8) * 4;
constexpr int kCastSmem = kCastStages * kCastStage;
__device__ __forceinline__ int cast_word(int row) { return row * kCastWords + (row >> 5) * 8; }

template <bool F32, bool COL, bool GROUPED>
__global__ void __launch_bounds__(kCastThreads, 2) mxfp4_cast_kernel(const CastParams p)
{
    constexpr int kSize = F32 ? 4 : 2;
    constexpr int kCols = 256 / kSize;        // columns of a tile
    constexpr int kPer = 32 / kSize;          // elements of a row that a thread holds
    constexpr int kHalves = F32 ? 2 : 1;      // tiles that share a 128-column scale tile
    extern __shared__ uint4 cast_smem[];
    __shared__ GroupTable<GROUPED> groups;
    pdl_wait_and_release();
    if (!GROUPED && p.noop != nullptr && *p.noop == 1.0f)
        return;
    const int tid = threadIdx.x;
    const int ct_all = p.col_tiles * kHalves;
    int64_t num_tiles = static_cast<int64_t>(p.row_tiles) * ct_all;
    if constexpr (GROUPED) {
        const int rt = group_setup<kCastThreads, kCastTile>(groups, p.offsets, p.num_groups, p.M);
        if (rt < 0) {
            if (blockIdx.x == 0 && tid == 0 && p.err_flag != nullptr)
                atomicOr(p.err_flag, 1);
            return;
        }
        num_tiles = static_cast<int64_t>(rt) * ct_all;
        clear_left_over<kCastThreads>(p.out_row, p.row_pitch, groups.offset[p.num_groups], p.M, p.rows, p.err_flag);
    }
    if (blockIdx.x >= num_tiles)
        return;
    const int count = static_cast<int>((num_tiles - 1 - blockIdx.x) / gridDim.x) + 1;
    const int nb = static_cast<int>((p.N + 31) / 32);
    const uint32_t smem = smem_u32(cast_smem);
    const void *nowhere = p.x != nullptr ? p.x : p.out_row;  // an address for copies of no bytes
    const int seg = tid & 7, r0 = tid >> 3;  // 32-byte piece, first of four rows 32 apart
    const int flip = seg >> 2;               // the last four pieces of a row go second half first: eight lanes, 32 banks

    struct Tile {
        int rt, ct;
        int64_t row0, row_end;
    };
    const int jump_rt = static_cast<int>(gridDim.x) / ct_all, jump_ct = static_cast<int>(gridDim.x) - jump_rt * ct_all;
    auto rows_of = [&](Tile &w) {
        w.row0 = static_cast<int64_t>(w.rt) * kCastTile;
        w.row_end = p.M;
        if constexpr (GROUPED) {
            const int g = groups.find(w.rt, p.num_groups);
            w.row0 = groups.offset[g] + static_cast<int64_t>(w.rt - groups.tile[g]) * kCastTile;
            w.row_end = groups.offset[g + 1];
        }
    };
    auto to_next = [&](Tile &w) {  // the CTA's next tile: gridDim.x tiles on
        w.ct += jump_ct;
        w.rt += jump_rt;
        if (w.ct >= ct_all) {
            w.ct -= ct_all;
            ++w.rt;
        }
        rows_of(w);
    };
    // The copies run a tile ahead of the casts, and the gathered rows' indices one tile ahead of the copies.
    Tile next;
    next.rt = static_cast<int>(blockIdx.x) / ct_all;
    next.ct = static_cast<int>(blockIdx.x) - next.rt * ct_all;
    rows_of(next);
    Tile at = next;
    int32_t index[4];
    auto fetch_indices = [&]() {
        if (GROUPED && p.rows != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t r = next.row0 + r0 + 32 * i;
                index[i] = r < next.row_end ? p.rows[r] : -1;
            }
        }
    };
    fetch_indices();
    uint32_t lost = 0;  // GROUPED: bits 4 s + i: row i of stage s names a row outside x
    int issued = 0;
    auto issue = [&]() {
        if (issued < count) {
            const int stage = issued % kCastStages;
            const uint32_t dst = smem + stage * kCastStage + seg * 32;
            const int64_t c = static_cast<int64_t>(next.ct) * kCols + seg * kPer;
            if (GROUPED)
                lost &= ~(0xFu << (4 * stage));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                int64_t from = next.row0 + r0 + 32 * i;
                bool live = from < next.row_end;
                if (GROUPED && live && p.rows != nullptr) {
                    from = index[i];
                    live = from >= 0 && from < p.T;
                    if (!live)
                        lost |= 1u << (4 * stage + i);
                }
                const unsigned char *src = static_cast<const unsigned char *>(p.x) + (from * p.ldx + c) * kSize;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int h = j ^ flip;
                    const bool ok = live && c + h * (kPer / 2) < p.N;  // N is a multiple of 8: a whole vector or none
                    copy16_async(dst + cast_word(r0 + 32 * i) * 4 + h * 16, ok ? src + h * 16 : nowhere, ok);
                }
            }
            if (++issued < count) {
                to_next(next);
                fetch_indices();
            }
        }
        copy_commit();
    };
    for (int s = 0; s < kCastStages - 1; ++s)
        issue();

    for (int n = 0; n < count; ++n) {
        copy_wait<kCastStages - 2>();
        if constexpr (COL)
            __syncthreads();  // tile n is there for every thread, and the stage before it free for the next copies
        const uint32_t gone = GROUPED ? lost >> (4 * (n % kCastStages)) : 0;
        issue();
        if (n > 0)
            to_next(at);
        const uint32_t *tile = reinterpret_cast<const uint32_t *>(reinterpret_cast<const unsigned char *>(cast_smem) + n % kCastStages * kCastStage);
        const int64_t col0 = static_cast<int64_t>(at.ct) * kCols;
        const int plane_ct = at.ct / kHalves, half = at.ct % kHalves;
        if (p.out_row != nullptr) {
            const int64_t c = col0 + seg * kPer;
            const bool in_blk = c / 32 < nb;
            unsigned char *out = p.out_row + (at.row0 + r0) * p.row_pitch + c / 2;
            uint8_t *sc_out = p.scale_row + (static_cast<int64_t>(at.rt) * p.col_tiles + plane_ct) * 512 + (r0 << 4);
            const int rows_left = static_cast<int>(at.row_end - at.row0 < kCastTile ? at.row_end - at.row0 : kCastTile);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 *q = reinterpret_cast<const uint4 *>(tile + cast_word(r0 + 32 * i) + seg * 8);  // this thread's own copies
                const uint4 q0 = q[flip], q1 = q[flip ^ 1];
                const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    m = F32 ? absmax_nan_f32(m, w[j]) : absmax_nan_bf16x2(m, w[j]);
                if (F32)
                    m &= 0x7FFFFFFFu;
                else
                    m = max(m << 16 & 0x7FFF0000u, m & 0x7FFF0000u);
                if (GROUPED && (gone >> i) & 1)
                    m = 0x7F800000u;
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                if (F32)
                    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                const int e = fp4_exponent(m);
                const uint64_t mul = f2_splat(fp4_multiplier(e));
                float v[kPer];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if constexpr (F32) {
                        v[j] = __uint_as_float(w[j]);
                    } else {
                        v[2 * j] = bf16_lo(w[j]);
                        v[2 * j + 1] = bf16_hi(w[j]);
                    }
                }
                const bool keep = r0 + 32 * i < rows_left && in_blk;
                if constexpr (F32) {
                    const uint32_t c8 = cvt_fp4x8_scaled(v, mul);
                    if (keep)
                        *reinterpret_cast<uint32_t *>(out) = e == 255 ? 0u : __funnelshift_l(c8, c8, 16 * flip);
                } else {
                    const uint32_t lo = e == 255 ? 0u : cvt_fp4x8_scaled(v, mul), hi = e == 255 ? 0u : cvt_fp4x8_scaled(v + 8, mul);
                    if (keep)
                        *reinterpret_cast<uint2 *>(out) = flip ? make_uint2(hi, lo) : make_uint2(lo, hi);
                }
                out += 32 * p.row_pitch;
                // the row's blocks, two (four) lanes apart, as the scale tile's 2 (4) bytes
                uint32_t sc = keep ? e : 0;
                sc |= __shfl_down_sync(0xFFFFFFFFu, sc, F32 ? 4 : 2) << 8;
                if (!F32)
                    sc |= __shfl_down_sync(0xFFFFFFFFu, sc, 4) << 16;
                if (seg == 0) {  // row r0 + 32 i: entry 16 r0 + 4 i
                    if constexpr (F32)
                        reinterpret_cast<uint16_t *>(sc_out + 4 * i)[half] = static_cast<uint16_t>(sc);
                    else
                        *reinterpret_cast<uint32_t *>(sc_out + 4 * i) = sc;
                }
                if (GROUPED && ((gone >> i) & 1) && at.ct == 0 && seg == 0 && p.err_flag != nullptr)
                    atomicOr(p.err_flag, 1);
            }
        }
        if constexpr (COL) {
            const int word = (tid >> 5) * 8 + (tid & 7), rb = (tid >> 3) & 3;  // word of the row, row block
            uint32_t w[32], m = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                w[i] = tile[cast_word(rb * 32 + i) + word];
                m = F32 ? absmax_nan_f32(m, w[i]) : absmax_nan_bf16x2(m, w[i]);
            }
            m &= F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
            const int64_t blk = at.row0 / 32 + rb;
            const bool live_blk = blk * 32 < p.M;
#pragma unroll
            for (int h = 0; h < (F32 ? 1 : 2); ++h) {
                const int e = fp4_exponent(F32 ? m : h ? m & 0xFFFF0000u : m << 16);
                const uint64_t mul = f2_splat(fp4_multiplier(e));
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t x = w[8 * q + j];
                        v[j] = F32 ? __uint_as_float(x) : h ? bf16_hi(x) : bf16_lo(x);
                    }
                    o[q] = e == 255 ? 0u : cvt_fp4x8_scaled(v, mul);
                }
                const int tc = F32 ? word : 2 * word + h;        // column of the tile
                const int lc = half * kCols + tc;                // column of the scale tile
                const bool keep = live_blk && col0 + tc < p.N;
                if (keep)
                    *reinterpret_cast<uint4 *>(p.out_col + (col0 + tc) * p.col_pitch + blk * 16) = make_uint4(o[0], o[1], o[2], o[3]);
                uint32_t sc = keep ? e : 0;  // the column's four blocks, eight lanes apart
                sc |= __shfl_down_sync(0xFFFFFFFFu, sc, 8) << 8;
                sc |= __shfl_down_sync(0xFFFFFFFFu, sc, 16) << 16;
                if (rb == 0)
                    *reinterpret_cast<uint32_t *>(p.scale_col + (static_cast<int64_t>(plane_ct) * p.row_tiles + at.rt) * 512 +
                                                  (((lc & 31) << 4) | ((lc >> 5) << 2))) = sc;
            }
        }
    }
    copy_wait<0>();
}

// Rows of a 4-bit matrix gathered for experts: codes row by row, scales into one plane per expert.  With more rows
// than tokens (each token goes to several experts) casting every token once and gathering 17/32 byte per element
// replaces a cast per row (65536 rows of 7168 from 8192 tokens: 251 -> 89 us, of which the gather 59).  A CTA takes 128 rows x 512 bytes of codes: a warp copies 16 rows, 16 bytes a lane.
struct GatherParams {
    const uint8_t *codes, *scale;  // of the T rows
    int64_t T, R, N;
    int64_t pitch;
    int col_tiles;
    const int32_t *rows;
    const int64_t *offsets;
    int num_groups;
    uint8_t *out, *out_scale;
    int *err_flag;
};
constexpr int kGatherTiles = 8;  // scale tiles of 64 code bytes per CTA

__global__ void __launch_bounds__(256, 5) mxfp4_gather_kernel(const GatherParams p)
{
    __shared__ GroupTable<true> groups;
    __shared__ int32_t index[kCastTile];
    pdl_wait_and_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row_tiles = group_setup<256, kCastTile>(groups, p.offsets, p.num_groups, p.R);
    if (row_tiles < 0) {
        if (blockIdx.x == 0 && tid == 0 && p.err_flag != nullptr)
            atomicOr(p.err_flag, 1);
        return;
    }
    clear_left_over<256>(p.out, p.pitch, groups.offset[p.num_groups], p.R, p.rows, p.err_flag);
    const int chunks = (p.col_tiles + kGatherTiles - 1) / kGatherTiles;
    const int nb = static_cast<int>((p.N + 31) / 32);
    const int64_t units = static_cast<int64_t>(row_tiles) * chunks;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int rt = static_cast<int>(u / chunks), chunk = static_cast<int>(u - static_cast<int64_t>(rt) * chunks);
        const int g = groups.find(rt, p.num_groups);
        const int64_t row0 = groups.offset[g] + static_cast<int64_t>(rt - groups.tile[g]) * kCastTile;
        const int64_t left = groups.offset[g + 1] - row0;
        const int valid = left < kCastTile ? static_cast<int>(left) : kCastTile;
        __syncthreads();  // the indices before are done with
        if (tid < valid) {
            int32_t i = p.rows[row0 + tid];
            if (i < 0 || i >= p.T) {
                i = -1;
                if (p.err_flag != nullptr)
                    atomicOr(p.err_flag, 1);
            }
            index[tid] = i;
        }
        __syncthreads();
        const int64_t byte = chunk * int64_t{kGatherTiles * 64} + lane * 16;
        if (byte < p.pitch) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 q[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = warp + 8 * (8 * h + j);
                    q[j] = make_uint4(0, 0, 0, 0);
                    if (r < valid && index[r] >= 0)
                        q[j] = __ldg(reinterpret_cast<const uint4 *>(p.codes + index[r] * p.pitch + byte));
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = warp + 8 * (8 * h + j);
                    if (r < valid)
                        *reinterpret_cast<uint4 *>(p.out + (row0 + r) * p.pitch + byte) = q[j];
                }
            }
        }
        const int r = tid & 127;
        const int32_t from = r < valid ? index[r] : -2;
#pragma unroll
        for (int j = 0; j < kGatherTiles / 2; ++j) {
            const int ct = chunk * kGatherTiles + (tid >> 7) + 2 * j;
            if (ct < p.col_tiles) {
                uint32_t v = 0;
                if (from >= 0)
                    v = *reinterpret_cast<const uint32_t *>(p.scale + ((static_cast<int64_t>(from) >> 7) * p.col_tiles + ct) * 512 + ((from & 31) << 4) +
                                                            (((from >> 5) & 3) << 2));
                else if (from == -1)  // NaN in the row's blocks, 0 past them
                    v = nb - 4 * ct >= 4 ? 0xFFFFFFFFu : (1u << (8 * (nb - 4 * ct))) - 1;
                *reinterpret_cast<uint32_t *>(p.out_scale + (static_cast<int64_t>(rt) * p.col_tiles + ct) * 512 + ((r & 31) << 4) + ((r >> 5) << 2)) = v;
            }
        }
    }
}

// Values of a 4-bit matrix.  A thread writes 16 aligned bytes (8 BF16 or 4 fp32) of each of several rows, whose codes
// and scales it loads first.  Where rows of the output are no whole vectors, its elements start at the row's first
// aligned one, anywhere in the codes.  Bound by its writes (8192x28672 to BF16 84 us, 7.1 TB/s; 7176x4093, off
// every boundary, 23 us, 3.2 TB/s, by issue).
template <bool VEC>
constexpr int kDecodeRows = VEC ? 8 : 4;  // a power of two: a thread's rows lie in one 32-row part of a scale tile

__device__ __forceinline__ float fp4_scale(uint32_t e)
{
    return e == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(e == 0 ? 0x400000u : e << 23);
}

// LONG: rows of 2^29 columns or more, whose scales lie 2^31 bytes and more apart: columns and their offsets in 64 bits (in
// 64 bits for every size, rows off vector boundaries took 3% longer to BF16 and 17% to fp32).
template <bool F32, bool VEC, bool LONG>
__global__ void __launch_bounds__(256) mxfp4_decode_kernel(const uint8_t *codes, const uint8_t *scale, int64_t rows, int64_t cols,
                                                           int64_t pitch, int64_t col_tiles, void *out)
{
    constexpr int V = F32 ? 4 : 8, kRows = kDecodeRows<VEC>, kSize = F32 ? 4 : 2;
    pdl_wait_and_release();
    const int64_t j = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;  // vector of the row
    using Col = std::conditional_t<LONG, int64_t, int>;
    const Col last = static_cast<Col>(cols) - 1;
    if (V * (j - 1) >= cols)  // off every row, whatever element its vectors start at
        return;
    const Col vj = static_cast<Col>(V * j);
    for (int64_t first = blockIdx.y * int64_t{kRows}; first < rows; first += int64_t{kRows} * gridDim.y) {
        const int n = static_cast<int>(rows - first < kRows ? rows - first : kRows);
        // the scale tile entry of (first, block 0): 16 bytes per row on; block b is b / 4 tiles and b % 4 bytes on
        const uint8_t *s = scale + (first >> 7) * col_tiles * 512 + ((first & 31) << 4) + (((first >> 5) & 3) << 2);
        const uint8_t *row = codes + first * pitch;
        // VEC: the row's column of every row's vector.  Else row i's vectors start (first + i) * cols % V elements early.
        const int lead0 = VEC ? 0 : static_cast<int>((first * cols) & (V - 1)), lead_step = VEC ? 0 : static_cast<int>(cols & (V - 1));
        uint32_t q[kRows], e0[kRows], e1[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int use = i < n ? i : n - 1;
            const Col c = vj - ((lead0 + use * lead_step) & (V - 1));
            if constexpr (VEC) {
                const Col at = c <= last ? max(c, Col{0}) : 0;
                q[i] = F32 ? *reinterpret_cast<const uint16_t *>(row + use * pitch + at / 2) : *reinterpret_cast<const uint32_t *>(row + use * pitch + at / 2);
                e0[i] = s[use * 16 + (at >> 7) * 512 + ((at >> 5) & 3)];
            } else {
                // the vector's elements from two words of codes and one or two blocks; past the ends any loaded value does
                const Col c0 = min(max(c, Col{0}), last), c1 = min(max(c0, c + V - 1), last);
                const uint32_t *words = reinterpret_cast<const uint32_t *>(row + use * pitch);
                // from before the row (c < 0) the first word is the upper one, and the lower one does not matter
                q[i] = __funnelshift_r(words[c0 >> 3], words[c1 >> 3], 4 * static_cast<int>(c & 7));
                e0[i] = s[use * 16 + (c0 >> 7) * 512 + ((c0 >> 5) & 3)];
                e1[i] = s[use * 16 + (c1 >> 7) * 512 + ((c1 >> 5) & 3)];
            }
        }
        unsigned char *to = static_cast<unsigned char *>(out) + (first * cols + V * j) * kSize;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (i >= n)
                break;
            const int lead = (lead0 + i * lead_step) & (V - 1);
            const Col c = vj - lead;
            unsigned char *dst = to + (i * cols - lead) * kSize;
            if (c > last)
                continue;
            const float m0 = fp4_scale(e0[i]), m1 = VEC ? m0 : fp4_scale(e1[i]);
            const int turn = VEC ? V : 32 - static_cast<int>(c & 31);  // elements of the first block
            float v[V];
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                fp4x2_to_f32((q[i] >> (8 * k)) & 0xFF, v[2 * k], v[2 * k + 1]);
                v[2 * k] *= 2 * k < turn ? m0 : m1;
                v[2 * k + 1] *= 2 * k + 1 < turn ? m0 : m1;
            }
            if (VEC || (c >= 0 && c + V - 1 <= last)) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)  // exact: the values have two significant bits
                    w[k] = F32 ? __float_as_uint(v[k]) : __byte_perm(__float_as_uint(v[(2 * k) % V]), __float_as_uint(v[(2 * k + 1) % V]), 0x7632);
                *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    if (c + k >= 0 && c + k <= last) {
                        if constexpr (F32)
                            reinterpret_cast<float *>(dst)[k] = v[k];
                        else
                            reinterpret_cast<uint16_t *>(dst)[k] = static_cast<uint16_t>(__float_as_uint(v[k]) >> 16);
                    }
                }
            }
        }
    }
}

}  // namespace mxfp8
