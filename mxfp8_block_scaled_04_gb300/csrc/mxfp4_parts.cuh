// Rows that are not cast, as exact operands of the MXFP4 products: x = sum of kParts 4-bit rows.
//
// Per block of 32, x * 2^k is rounded to an integer X of 24 bits, with k such that the block's largest magnitude amax becomes at
// least 1.71 * 2^21: an error of at most 2^-22.7 amax per element (2^-128 where the blocks' values are so small that k would
// pass 127).  X has eight octal digits, balanced between -4 and 3, which E2M1 holds exactly; part j is the digits of weight
// 8^(7 - j), with the scale 2^(21 - 3j - k).  X + 4 * (8^8 - 1) / 7 has the digits plus 4 as its octal digits, so that all of
// this is shifts and logic: a digit of eight elements at a time.  (Casting what the parts before leave, with the conversion
// instructions, took three times as long.)  The parts are rows 8i to 8i + 7 of the tokens' operand: one token fills half of
// the smallest MMA's 16 columns, sixteen fill 128, and the weights' bytes remain the time.  The products' epilogue adds a
// row's eight sums in fp32, the smallest first.
//
// A warp takes 256 columns of a row: four lanes share a block, each with 8 elements.  Bound by launch and latency for the
// few rows that this serves.
#pragma once

#include <cstdint>

#include "groups.cuh"
#include "mxfp4_cast.cuh"
#include "ptx.cuh"

namespace mxfp8 {

constexpr int kParts = 8;
// A thread takes 8 columns of a row.  Grouped, two CTAs of 256 threads per SM, whose tables of groups leave the shared memory
// that a CTA of the products needs to start beside them (16 tokens to 8 of 64 experts, 7168 -> 2048, over the products' own 69
// us: 11 us without that limit, 7.2 with it; 64 tokens 22, with CTAs of 128 threads 27).
template <bool GROUPED>
constexpr int kPartsThreads = GROUPED ? 256 : 128;
constexpr int kPartsGroupedCtas = 2;

struct PartsParams {
    const void *x;
    int64_t T, R, K, ldx;        // rows of x, rows of the operand (before parts), columns, pitch
    uint8_t *out, *scale;
    int64_t pitch;               // bytes of a row of codes
    int col_tiles, chunks;       // scale tiles along K, CTAs along K
    const int32_t *rows;         // grouped
    const int64_t *offsets;
    int num_groups;
    int *err_flag;
};

// E2M1 codes of eight balanced octal digits plus 4, one to four bits of w: 0 .. 7 stand for -4 .. 3, whose codes are
// 14, 13, 12, 10, 0, 2, 4, 5.
__device__ __forceinline__ uint32_t digit_codes(uint32_t w)
{
    constexpr uint32_t kOnes = 0x11111111u;
    const uint32_t b0 = w, b1 = w >> 1, b2 = w >> 2;
    const uint32_t c2 = (b2 & b1) | (~b2 & ~(b1 & b0));
    const uint32_t c1 = (b2 & ~b1 & b0) | (~b2 & ~(b1 ^ b0));
    const uint32_t c0 = (b2 & b1 & b0) | (~b2 & ~b1 & b0);
    return (c0 & kOnes) | (c1 & kOnes) << 1 | (c2 & kOnes) << 2 | (~b2 & kOnes) << 3;
}

// Eight elements of x split into parts: put(j, codes of part j, scale bytes of part j for the four blocks from lane & ~15 on).
// All lanes of the warp, four to a block; `live` false: a row that x does not have.  A block that holds a NaN or an infinity,
// like such a row, gets the scale 255 in part 0 and zero codes.
template <typename Put>
__device__ __forceinline__ void split_parts(const float (&v)[8], bool live, Put &&put)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);  // as integers a NaN lies above every number
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const bool nan = !live || m >= 0x7F800000u;
    // 2^k: 22 - exponent, one less for a mantissa above 1.71 (digits of at most 3 reach 0.857 * 2^23)
    const int e = max(static_cast<int>(m >> 23) - 1 + ((m & 0x7FFFFFu) > 0x5B0000u ? 1 : 0), 21);  // 148 - k, part 0's scale
    const float mul = __uint_as_float(static_cast<uint32_t>(nan ? 0 : 275 - e) << 23);
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        u[i] = 0x924924u + static_cast<uint32_t>(nan ? 0 : __float2int_rn(v[i] * mul));
    uint32_t scales = static_cast<uint32_t>(nan ? 255 : e);
    scales |= __shfl_down_sync(0xFFFFFFFFu, scales, 4) << 8;  // four blocks, four lanes apart
    scales |= __shfl_down_sync(0xFFFFFFFFu, scales, 8) << 16;
#pragma unroll
    for (int j = 0; j < kParts; ++j) {
        const int down = 21 - 3 * j;
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w |= (4 * i >= down ? u[i] << (4 * i - down) : u[i] >> (down - 4 * i)) & (7u << (4 * i));
        put(j, digit_codes(w), scales);
        scales -= 0x03030303u;  // every byte is at least 21
    }
}

template <bool F32, bool GROUPED>
__global__ void __launch_bounds__(kPartsThreads<GROUPED>) mxfp4_parts_kernel(const PartsParams p)
{
    constexpr int kThreads = kPartsThreads<GROUPED>;
    __shared__ GroupTable<GROUPED> groups;
    pdl_wait_and_release();  // in this order: the products' kernel reads weights and offsets as soon as it is let start
    const int tid = threadIdx.x, lane = tid & 31;
    // A unit's elements are loaded before the one before it is split, the first ones before the table of groups is made.
    struct Unit {
        uint4 lo, hi;
        bool live;  // the row is one of x's
    };
    auto fetch = [&](int64_t u) {
        Unit n{};
        const int64_t i = u / p.chunks;
        if (i >= p.R)
            return n;
        const int64_t c = (u - i * p.chunks) * (8 * kThreads) + tid * 8;
        int64_t from = i;
        n.live = true;
        if (GROUPED && p.rows != nullptr) {
            from = p.rows[i];
            n.live = from >= 0 && from < p.T;
        }
        if (n.live && c < p.K) {  // K is a multiple of 8
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(p.x) + (from * p.ldx + c) * (F32 ? 4 : 2));
            n.lo = src[0];
            if constexpr (F32)
                n.hi = src[1];
        }
        return n;
    };
    Unit next = fetch(blockIdx.x);
    if constexpr (GROUPED) {
        const int rt = group_setup<kThreads, kCastTile, kParts>(groups, p.offsets, p.num_groups, p.R * kParts);
        if (rt < 0) {
            if (blockIdx.x == 0 && tid == 0 && p.err_flag != nullptr)
                atomicOr(p.err_flag, 1);
            return;
        }
        const int64_t end = groups.offset[p.num_groups] / kParts;  // rows past it belong to no expert: a plan marks them
        bool lost = false;
        for (int64_t r = end + blockIdx.x * int64_t{kThreads} + tid; r < p.R; r += gridDim.x * int64_t{kThreads})
            lost |= p.rows == nullptr || p.rows[r] >= 0;
        if (lost && p.err_flag != nullptr)
            atomicOr(p.err_flag, 1);
    }
    int64_t all = p.R;
    if constexpr (GROUPED)
        all = groups.offset[p.num_groups] / kParts;
    const int64_t units = all * p.chunks;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t i = u / p.chunks;
        const int64_t c = (u - i * p.chunks) * (8 * kThreads) + tid * 8;
        int64_t tile0 = 0, r0 = i * kParts;
        const Unit at = next;
        next = fetch(u + gridDim.x);
        if constexpr (GROUPED) {
            if (!at.live && tid == 0 && p.err_flag != nullptr)
                atomicOr(p.err_flag, 1);
            int lo = 0, hi = p.num_groups;  // the last group that starts at or before the row (those before it may be empty)
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (groups.offset[mid] <= r0)
                    lo = mid;
                else
                    hi = mid;
            }
            tile0 = groups.plane[lo];
            r0 -= groups.offset[lo];
        }
        float v[8];
        if constexpr (F32) {
            const uint32_t w[8] = {at.lo.x, at.lo.y, at.lo.z, at.lo.w, at.hi.x, at.hi.y, at.hi.z, at.hi.w};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = __uint_as_float(w[j]);
        } else {
            const uint32_t w[4] = {at.lo.x, at.lo.y, at.lo.z, at.lo.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = bf16_lo(w[j]);
                v[2 * j + 1] = bf16_hi(w[j]);
            }
        }
        const int64_t blk = c / 32;
        const bool in_row = c < p.pitch * 2;  // a row's last block is written whole
        const int64_t r = r0;
        uint8_t *codes = p.out + i * kParts * p.pitch + c / 2;
        uint8_t *tile = p.scale + ((tile0 + (r >> 7)) * p.col_tiles + blk / 4) * 512 + ((r & 31) << 4) + (((r >> 5) & 3) << 2);
        split_parts(v, at.live, [&](int j, uint32_t q, uint32_t scales) {  // (rows 8i .. 8i + 7 lie in one 32-row part of a scale tile)
            if (in_row)
                *reinterpret_cast<uint32_t *>(codes + j * p.pitch) = q;
            if ((lane & 15) == 0 && blk / 4 < p.col_tiles)
                *reinterpret_cast<uint32_t *>(tile + j * 16) = scales;
        });
    }
}

}  // namespace mxfp8
