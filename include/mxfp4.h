/*
 * mxfp4.h -- C ABI of the MXFP4 (4-bit microscaled) cast and products, same library as mxfp8.h.
 *
 * A block of 32 consecutive elements shares one E8M0 scale; each element is E2M1 (1 sign, 2 exponent,
 * 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).  Per block, with amax = max |x|:
 *     e = clamp(ceil(log2(amax / 6)) + 127, 0, 254)        (amax == 0 -> e = 127)
 *     q = round-to-nearest-even to E2M1 of x * 2^(127 - e) (never above 6: nothing saturates)
 * the rule of the MXFP8 cast with Fmax = 6.  A block that holds a NaN or an infinity gets the E8M0 NaN
 * (255) and zero codes: every element of it decodes to NaN, and so does every product that reads it.
 *
 * A 4-bit matrix of R rows and C columns (blocks along the columns) is
 *     codes   uint8 [R, mxfp4_row_bytes(C)]: element 2i in the low half of byte i; a row's last block is
 *             padded with zero codes (any C; row_bytes is 16 per block);
 *     scales  one plane of mxfp4_scale_bytes(R, C) bytes, GEMM-ready (MXFP8_SCALES_SWIZZLED): tiles of
 *             128 rows x 4 blocks, row-tile major, entry (r, b) of a tile at
 *             16 * (r % 32) + 4 * (r / 32) + b.  The cast writes every byte; those past R or past
 *             ceil(C / 32) are 0.  (In a plane from elsewhere those past ceil(C / 32) may hold anything but 255.)
 * The conventions of mxfp8.h hold for every call here: the caller's buffers, host-side checks that return a
 * status, work ordered on `stream` and launched with programmatic stream serialization, nothing read on
 * the host, no allocation.
 */
#ifndef MXFP4_GB300_H
#define MXFP4_GB300_H

#include <stddef.h>
#include <stdint.h>

#include "mxfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of unquantized inputs and outputs. */
typedef enum {
    MXFP4_BF16 = 0,
    MXFP4_F32 = 1
} mxfp4_type_t;

/* Bytes of one row of codes: 16 * ceil(cols / 32).  0 for cols <= 0. */
size_t mxfp4_row_bytes(int64_t cols);

/* Bytes of the scale plane of a [rows, cols] matrix: 512 * ceil(rows / 128) * ceil(cols / 128). */
size_t mxfp4_scale_bytes(int64_t rows, int64_t cols);

/*
 * Cast x [M, N] (row pitch ldx elements), once along its rows and once, transposed, along its columns.
 *
 *   x            device, x_type, 16-byte aligned; N and ldx multiples of 8, ldx >= N.
 *   out_row, scale_row   the matrix [M, N]; both NULL skips it.
 *   out_col, scale_col   its transpose as a matrix [N, M] (blocks of 32 rows of x; rows past M count as
 *                zeros): the operand layout of the products that sum over M.  Both NULL skips it.
 *                out_* 16-byte aligned, scale_* 4-byte aligned (16 for the products).
 *   noop         device fp32 scalar or NULL: when *noop == 1.0f nothing is written.
 *
 * MXFP8_ERR_FORMAT (x_type), _SHAPE, _NULL (a half-set pair, no direction, x), _ALIGN, _DEVICE, _LAUNCH.
 * M == 0 or N == 0: nothing to do.
 */
mxfp8_status_t mxfp4_quantize(const void *x, int x_type, int64_t M, int64_t N, int64_t ldx, void *out_row,
                              void *scale_row, void *out_col, void *scale_col, const float *noop, void *stream);

/*
 * Bytes that hold the scale planes of a grouped cast of total_rows rows, whatever the offsets: every
 * group's plane is padded to whole 128-row tiles, (total_rows / 128 + min(num_groups, total_rows)) row
 * tiles at most.
 */
size_t mxfp4_grouped_scale_bytes(int64_t total_rows, int64_t cols, int num_groups);

/*
 * The rowwise cast of rows gathered for experts: output row i is the cast of x row rows[i] (or of row i
 * when rows is NULL, then total_rows <= T), and rows [offsets[g], offsets[g+1]) belong to expert g.
 * out [total_rows, row_bytes(N)]; `scale` holds one GEMM-ready plane per expert (rows_g x N), each on its
 * own, one after the other (mxfp4_grouped_scale_bytes(total_rows, N, num_groups) bytes are enough).
 *
 *   x            device, x_type, [T, N], row pitch ldx.
 *   rows         device int32 [total_rows] or NULL.  An index outside [0, T) reads nothing: its row
 *                becomes NaN scales, and *err_flag (if given) is set to 1.
 *   offsets      device int64 [num_groups + 1] from 0, non-decreasing, none above total_rows, else nothing
 *                is written and *err_flag is set to 1.  1 <= num_groups <= MXFP8_MAX_GROUPS.
 *                Rows from offsets[num_groups] to total_rows belong to no expert (the choices that a plan
 *                drops): their codes are zeros.  Where `rows` does not mark such a row with a negative index,
 *                as a plan does, and where there are such rows without `rows`, *err_flag is set to 1 too.
 *   err_flag     device int or NULL, never cleared here.
 *   workspace    NULL, or device memory of mxfp4_quantize_grouped_workspace_bytes(T, N, total_rows) bytes,
 *                16-byte aligned: with it, a gather of more rows than T casts every row of x once and gathers
 *                the codes, to the same result (measured 3 times faster at 8 rows per token).
 */
mxfp8_status_t mxfp4_quantize_grouped(const void *x, int x_type, int64_t T, int64_t N, int64_t ldx, const int32_t *rows,
                                      int64_t total_rows, int num_groups, const int64_t *offsets, void *out,
                                      void *scale, int *err_flag, void *workspace, void *stream);

/* 0 unless total_rows > T. */
size_t mxfp4_quantize_grouped_workspace_bytes(int64_t T, int64_t N, int64_t total_rows);

/*
 * The values of a 4-bit matrix: out [rows, cols] (row pitch cols, any cols up to 2^31 - 1) in out_type.  Exact in
 * both types, but for 2^128, which an element of at least 1.75 * 2^127 rounds up to: it comes out as infinity.
 */
mxfp8_status_t mxfp4_dequantize(const void *codes, const void *scale, int64_t rows, int64_t cols, void *out,
                                int out_type, void *stream);

/*
 * out [M, N] = A [M, K] * B [N, K]^T for 4-bit matrices A and B, products exact, sums in fp32, rounded once
 * to out_type.  Forward, input gradient and weight gradient of a linear layer are all this call: y = x W^T,
 * dx = dy (W^T)^T with W's transposed cast, dw = (dy^T) (x^T)^T with both transposed casts.
 *
 *   codes 16-byte aligned, scale planes 16-byte aligned, out aligned to its element; ldo >= N elements.
 *   M, N, K any size from 0 to 2^31 - 1 (K = 0: out is set to zeros).
 */
mxfp8_status_t mxfp4_matmul(const void *a_codes, const void *a_scale, int64_t M, const void *b_codes,
                            const void *b_scale, int64_t N, int64_t K, void *out, int out_type, int64_t ldo,
                            void *stream);

/*
 * The experts' products in one launch: rows [offsets[g], offsets[g+1]) of out [total_rows, N] are those rows
 * of A (a grouped cast; a_scale of mxfp4_grouped_scale_bytes(total_rows, K, num_groups) bytes) times B_g^T.
 * b_codes [num_groups, N, row_bytes(K)]; b_scale [num_groups] planes of mxfp4_scale_bytes(N, K).  offsets as for
 * mxfp4_quantize_grouped; rows of no expert become zeros, and *err_flag (if given) is set to 1 where there are any: with a
 * plan that drops choices, the flag of the gathered cast is the one that tells a fault from a dropped choice.
 */
mxfp8_status_t mxfp4_matmul_grouped(const void *a_codes, const void *a_scale, int64_t total_rows, int num_groups,
                                    const int64_t *offsets, const void *b_codes, const void *b_scale, int64_t N,
                                    int64_t K, void *out, int out_type, int *err_flag, void *stream);

/*
 * Products of rows that are not cast with 4-bit weights (serving: weights in 4 bits, tokens as they are):
 * out [M, N] = x [M, K] * B [N, K]^T, sums in fp32, rounded once to out_type.  x enters as a sum of eight 4-bit rows per row,
 * 24-bit fixed point under each block's scale: an element differs from x by at most 2^-22 of the largest magnitude in its block of
 * 32 (or 2^-126).  Where a block's magnitudes are alike that is fp32 accuracy; an element 2^-15 of its block's largest keeps about
 * 8 bits, one below 2^-23 hardly any.  What the parts add up to on the way is at most 7/3 of sum |x| |B|: where that passes fp32's range
 * the result may be an infinity or NaN though x and the result do not.  A NaN or an infinity in a row of x makes that output row
 * NaN.
 *
 *   x            device, x_type, 16-byte aligned; K and ldx multiples of 8, ldx >= K; M < 2^28.
 *   b_codes, b_scale, out, out_type, ldo   as for mxfp4_matmul.  (A block of B with scale 255 makes its output column NaN.)
 *   workspace    device, mxfp4_linear_workspace_bytes(M, K, N) bytes (0 for few rows, two at least: NULL), 16-byte aligned; not
 *                shared by calls that may overlap.
 *
 * Meant for few rows (the weights' bytes are the time up to about 16; every row costs eight of the tensor cores' columns):
 * for many, cast x and call mxfp4_matmul.
 */
size_t mxfp4_linear_workspace_bytes(int64_t M, int64_t K, int64_t N);

mxfp8_status_t mxfp4_linear(const void *x, int x_type, int64_t M, int64_t K, int64_t ldx, const void *b_codes,
                            const void *b_scale, int64_t N, void *out, int out_type, int64_t ldo, void *workspace,
                            void *stream);

/*
 * The same for experts: row i of out [total_rows, N] is x row rows[i] (row i when rows is NULL, then total_rows <= T) times
 * B_g^T of the expert g whose rows [offsets[g], offsets[g+1]) it is in.  rows, offsets and err_flag as for
 * mxfp4_quantize_grouped (an index outside x: a row of NaN; rows past the last offset: zeros, and *err_flag is set where
 * `rows` does not mark them with a negative index; bad offsets: nothing is written).  b_codes, b_scale as for
 * mxfp4_matmul_grouped.  workspace: mxfp4_linear_grouped_workspace_bytes(total_rows, K, num_groups) bytes (0 for few rows on
 * many experts: NULL).
 */
size_t mxfp4_linear_grouped_workspace_bytes(int64_t total_rows, int64_t K, int num_groups);

mxfp8_status_t mxfp4_linear_grouped(const void *x, int x_type, int64_t T, int64_t K, int64_t ldx, const int32_t *rows,
                                    int64_t total_rows, int num_groups, const int64_t *offsets, const void *b_codes,
                                    const void *b_scale, int64_t N, void *out, int out_type, int *err_flag,
                                    void *workspace, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MXFP4_GB300_H */
