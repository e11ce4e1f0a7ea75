// MXFP4 cast and its inverse (sm_103a); formulas and layouts in include/mxfp4.h.
//
// One pass over HBM.  A CTA takes a 128x128 tile: its rows' and its columns' scales are then one 512-byte
// tile of each GEMM-ready plane.  Rowwise, a thread holds 16 consecutive elements of a row and a block is two
// lanes; columnwise, the tile goes through shared memory and a thread takes two neighbouring columns of 32
// rows, so that the four lanes of a column write 64 consecutive bytes of the transposed codes.  Bound by HBM:
// 2 (or 4) bytes in and 17/32 byte out per element and direction.
//
// The scale exponent comes from the bits of amax (exact), x * 2^(127 - e) is exact wherever the rounding to
// E2M1 depends on it (powers of two, fp32 subnormals kept), so the codes are those of the definition.
#pragma once

#include <cstdint>

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

// Two E2M1 codes (a byte) -> two fp32.
__device__ __forceinline__ void fp4x2_to_f32(uint32_t byte, float &lo, float &hi)
{
    uint32_t h;
    asm("{\n\t.reg .b8 b, z0, z1, z2;\n\tmov.b32 {b, z0, z1, z2}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(lo), "=f"(hi) : "r"(h));
}

// 16 consecutive elements of a row in registers: 8 words of BF16 pairs, or 16 fp32.
template <bool F32>
struct Seg {
    uint32_t w[F32 ? 16 : 8];
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (F32)
            return __uint_as_float(w[i]);
        else
            return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    }
    // fp32 bits of max |x|
    __device__ __forceinline__ uint32_t amax() const
    {
        uint32_t m = 0;
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                m = max(m, w[i] & 0x7FFFFFFFu);
            return m;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = max_u16x2(m, w[i] & 0x7FFF7FFFu);
            return max(m & 0xFFFFu, m >> 16) << 16;
        }
    }
};

// Shared memory of the columnwise direction: rows of 128 elements, each group of 32 rows shifted by a
// quarter of the banks, so that a warp's reads of 8 column pairs x 4 row blocks hit 32 banks.
template <bool F32>
constexpr int kCastWords = F32 ? 128 : 64;
template <bool F32>
__host__ __device__ constexpr int cast_smem_bytes(bool col)
{
    return col ? (kCastTile * kCastWords<F32> + 3 * kCastWords<F32> / 8) * 4 : 0;
}

template <bool F32, bool COL, bool GROUPED>
__global__ void __launch_bounds__(kCastThreads) mxfp4_cast_kernel(const CastParams p)
{
    extern __shared__ uint4 cast_smem[];
    __shared__ uint32_t sc_row[kCastTile], sc_col[kCastTile];  // one plane tile each, as its 4-byte entries
    __shared__ GroupTable<GROUPED> groups;
    pdl_wait_and_release();
    if (!GROUPED && p.noop != nullptr && *p.noop == 1.0f)
        return;
    const int tid = threadIdx.x;
    int num_tiles = p.row_tiles * p.col_tiles;
    if constexpr (GROUPED) {
        const int rt = group_setup<kCastThreads, kCastTile>(groups, p.offsets, p.num_groups, p.M);
        if (rt < 0) {
            if (blockIdx.x == 0 && tid == 0 && p.err_flag != nullptr)
                atomicOr(p.err_flag, 1);
            return;
        }
        num_tiles = rt * p.col_tiles;
    }
    const int nb = static_cast<int>((p.N + 31) / 32);
    uint32_t *tile = reinterpret_cast<uint32_t *>(cast_smem);
    constexpr int W = kCastWords<F32>;
    constexpr int V = F32 ? 4 : 2;  // 16-byte loads per segment

    for (int t = blockIdx.x; t < num_tiles; t += gridDim.x) {
        const int rt = t / p.col_tiles, ct = t - rt * p.col_tiles;
        int64_t row0 = static_cast<int64_t>(rt) * kCastTile, row_end = p.M;
        if constexpr (GROUPED) {
            const int g = groups.find(rt, p.num_groups);
            row0 = groups.offset[g] + static_cast<int64_t>(rt - groups.tile[g]) * kCastTile;
            row_end = groups.offset[g + 1];
        }
        const int64_t col0 = static_cast<int64_t>(ct) * kCastTile;
        const int seg = tid & 7, r0 = tid >> 3;
        const int64_t c = col0 + seg * 16;
        const int valid = c >= p.N ? 0 : p.N - c >= 16 ? 16 : 8;  // N is a multiple of 8

        Seg<F32> s[4];
        bool bad[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = row0 + r0 + 32 * i;
            bool live = r < row_end;
            int64_t src = r;
            bad[i] = false;
            if (GROUPED && live && p.rows != nullptr) {
                src = p.rows[r];
                if (src < 0 || src >= p.T) {
                    live = false;
                    bad[i] = true;
                }
            }
            const uint4 *g = reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(p.x) + (src * p.ldx + c) * (F32 ? 4 : 2));
#pragma unroll
            for (int v = 0; v < V; ++v) {
                uint4 q = make_uint4(0, 0, 0, 0);
                if (live && v * (16 / V) < valid)
                    q = __ldg(g + v);
                s[i].w[4 * v] = q.x;
                s[i].w[4 * v + 1] = q.y;
                s[i].w[4 * v + 2] = q.z;
                s[i].w[4 * v + 3] = q.w;
            }
        }
        if constexpr (COL) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t *d = tile + (r0 + 32 * i) * W + i * (W / 8) + seg * (W / 8);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    reinterpret_cast<uint4 *>(d)[v] = make_uint4(s[i].w[4 * v], s[i].w[4 * v + 1], s[i].w[4 * v + 2], s[i].w[4 * v + 3]);
            }
        }
        if (p.out_row != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int lr = r0 + 32 * i;
                const int64_t r = row0 + lr;
                uint32_t m = bad[i] ? 0x7F800000u : s[i].amax();
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                const int e = fp4_exponent(m);
                const float mul = fp4_multiplier(e);
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j] = s[i].get(j) * mul;
                uint32_t lo = cvt_fp4x8(v), hi = cvt_fp4x8(v + 8);
                if (e == 255)
                    lo = hi = 0;
                const int64_t blk = c / 32;
                if (r < row_end && blk < nb)
                    *reinterpret_cast<uint2 *>(p.out_row + r * p.row_pitch + c / 2) = make_uint2(lo, hi);
                if ((seg & 1) == 0)
                    reinterpret_cast<uint8_t *>(sc_row)[((lr & 31) << 4) | ((lr >> 5) << 2) | (seg >> 1)] =
                        static_cast<uint8_t>(r < row_end && blk < nb ? e : 0);
                if (GROUPED && bad[i] && ct == 0 && seg == 0 && p.err_flag != nullptr)
                    atomicOr(p.err_flag, 1);
            }
        }
        if (COL || p.out_row != nullptr)
            __syncthreads();
        if (p.out_row != nullptr && tid < kCastTile)
            reinterpret_cast<uint32_t *>(p.scale_row)[static_cast<int64_t>(t) * kCastTile + tid] = sc_row[tid];
        if constexpr (COL) {
            const int cp = (tid >> 5) * 8 + (tid & 7), rb = (tid >> 3) & 3;  // column pair, row block
            uint32_t m0 = 0, m1 = 0;
            uint32_t w0[32], w1[F32 ? 32 : 1];
            if constexpr (F32) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const uint2 q = *reinterpret_cast<const uint2 *>(tile + (rb * 32 + i) * W + rb * (W / 8) + 2 * cp);
                    w0[i] = q.x;
                    w1[i] = q.y;
                    m0 = max(m0, q.x & 0x7FFFFFFFu);
                    m1 = max(m1, q.y & 0x7FFFFFFFu);
                }
            } else {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    w0[i] = tile[(rb * 32 + i) * W + rb * (W / 8) + cp];
                    m = max_u16x2(m, w0[i] & 0x7FFF7FFFu);
                }
                m0 = m << 16;
                m1 = m & 0xFFFF0000u;
            }
            const int64_t blk = row0 / 32 + rb;
            const bool live_blk = blk * 32 < p.M;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int e = fp4_exponent(h ? m1 : m0);
                const float mul = fp4_multiplier(e);
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t w = w0[8 * q + j];
                        float f;
                        if constexpr (F32)
                            f = __uint_as_float(h ? w1[8 * q + j] : w);
                        else
                            f = h ? bf16_hi(w) : bf16_lo(w);
                        v[j] = f * mul;
                    }
                    o[q] = e == 255 ? 0u : cvt_fp4x8(v);
                }
                const int lc = 2 * cp + h;
                const bool live = live_blk && col0 + lc < p.N;
                if (live)
                    *reinterpret_cast<uint4 *>(p.out_col + (col0 + lc) * p.col_pitch + blk * 16) = make_uint4(o[0], o[1], o[2], o[3]);
                reinterpret_cast<uint8_t *>(sc_col)[((lc & 31) << 4) | ((lc >> 5) << 2) | rb] = static_cast<uint8_t>(live ? e : 0);
            }
            __syncthreads();
            if (tid < kCastTile)
                reinterpret_cast<uint32_t *>(p.scale_col)[(static_cast<int64_t>(ct) * p.row_tiles + rt) * kCastTile + tid] = sc_col[tid];
        }
        if (t + static_cast<int>(gridDim.x) < num_tiles)
            __syncthreads();  // the next tile reuses the shared arrays
    }
}

// Values of a 4-bit matrix.  A thread writes 8 elements of a row: 16 or 32 bytes at once where rows of the output
// are whole vectors (VEC, cols a multiple of 8), one by one otherwise.  Bound by its writes.
template <bool F32, bool VEC>
__global__ void __launch_bounds__(256) mxfp4_decode_kernel(const uint8_t *codes, const uint8_t *scale, int64_t rows, int64_t cols,
                                                           int64_t pitch, int64_t col_tiles, void *out)
{
    pdl_wait_and_release();
    const int64_t per_row = (cols + 7) / 8, n = rows * per_row;
    for (int64_t i = blockIdx.x * int64_t{256} + threadIdx.x; i < n; i += int64_t{256} * gridDim.x) {
        const int64_t r = i / per_row, c = (i - r * per_row) * 8;
        const uint32_t q = *reinterpret_cast<const uint32_t *>(codes + r * pitch + c / 2);
        const int64_t blk = c / 32;
        const uint32_t e = scale[((r >> 7) * col_tiles + (blk >> 2)) * 512 + ((r & 31) << 4) + (((r >> 5) & 3) << 2) + (blk & 3)];
        const float mul = e == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(e == 0 ? 0x400000u : e << 23);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            fp4x2_to_f32((q >> (8 * j)) & 0xFF, v[2 * j], v[2 * j + 1]);
            v[2 * j] *= mul;
            v[2 * j + 1] *= mul;
        }
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)  // exact: the values have two significant bits
            w[j] = (__float_as_uint(v[2 * j]) >> 16) | (__float_as_uint(v[2 * j + 1]) & 0xFFFF0000u);
        if constexpr (!VEC) {
            for (int j = 0; j < 8 && c + j < cols; ++j) {
                if constexpr (F32)
                    static_cast<float *>(out)[r * cols + c + j] = v[j];
                else
                    static_cast<uint16_t *>(out)[r * cols + c + j] = static_cast<uint16_t>(__float_as_uint(v[j]) >> 16);
            }
        } else if constexpr (F32) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + r * cols + c);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + r * cols + c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

}  // namespace mxfp8
