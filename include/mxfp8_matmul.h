/*
 * mxfp8_matmul.h -- C ABI of the experts' products in MXFP8, same library as mxfp8.h, whose conventions hold here (the
 * caller's buffers, status codes, stream order, no allocation, nothing read on the host).
 *
 * The operands are the outputs of mxfp8_quantize_grouped_swizzled as they are: FP8 codes row-major, and GEMM-ready
 * scale planes, one per expert, one after the other.  An expert layer with weights W [E, N, K] and rows x [R, K] sorted
 * by expert (offsets: expert g owns rows [offsets[g], offsets[g+1])) has three products:
 *     forward           y  [R, N] = x W_g^T     x's rows and W's rows        (blocks of 32 along K)
 *     input gradient    dx [R, K] = dy W_g      dy's rows and W's columns    (blocks of 32 along N)
 *     weight gradient   dW_g [N, K] = dy_g^T x_g   dy's and x's columns      (blocks of 32 rows of the expert)
 * W is the cast of its [E * N, K] rows in E groups of N rows.  Products of codes and scales are exact, sums fp32, rounded
 * once to the output's type.  Sums to fp32 are made in pieces (2048 rows of a weight gradient, 8192 elements of the other two)
 * that are added in order: the tensor core truncates its sums.  Formats may differ between the operands (MXFP8_E4M3, MXFP8_E5M2).
 */
#ifndef MXFP8_MATMUL_GB300_H
#define MXFP8_MATMUL_GB300_H

#include <stddef.h>
#include <stdint.h>

#include "mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Which of the three products. */
typedef enum {
    MXFP8_FORWARD = 0,
    MXFP8_INPUT_GRADIENT = 1,
    MXFP8_WEIGHT_GRADIENT = 2
} mxfp8_product_t;

/*
 * One product of all experts in one launch.
 *
 *   a, a_scale, a_scale_bytes, a_fmt   forward: out_row, scale_row of x [R, K]; input gradient: out_row, scale_row of
 *                dy [R, N]; weight gradient: out_col, scale_col of dy [R, N].  The bytes are the plane's size; offsets
 *                that need more are bad offsets.
 *   b, b_scale, b_scale_bytes, b_fmt   forward: out_row, scale_row of W; input gradient: out_col, scale_col of W; weight
 *                gradient: out_col, scale_col of x [R, K].
 *   N, K         multiples of 16 (a TMA row), below 2^31; num_groups * N < 2^31.
 *   out          forward [R, N], input gradient [R, K], weight gradient [num_groups, N, K] (zeros for an expert without
 *                rows), MXFP4_BF16 or MXFP4_F32, 16-byte aligned.
 *   offsets      device int64 [num_groups + 1] from 0, non-decreasing, none above R, else nothing is written and *err_flag
 *                is set to 1.  Rows from offsets[num_groups] to R belong to no expert: forward and input gradient write
 *                zeros there, the weight gradient leaves them out, and *err_flag is set to 1 too.
 *   err_flag     device int or NULL, never cleared here.
 *   codes and planes 16-byte aligned.  A plane's bytes past an expert's rows or blocks may be anything but 255.
 *
 * MXFP8_ERR_FORMAT (product, formats, out_type), _SHAPE, _GROUPS, _NULL, _ALIGN, _WORKSPACE (W's plane too small), _DEVICE,
 * _LAUNCH.
 */
mxfp8_status_t mxfp8_matmul_grouped(int product, const void *a, const void *a_scale, size_t a_scale_bytes, int a_fmt,
                                    const void *b, const void *b_scale, size_t b_scale_bytes, int b_fmt,
                                    int64_t total_rows, int64_t N, int64_t K, int num_groups, const int64_t *offsets,
                                    void *out, int out_type, int *err_flag, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MXFP8_MATMUL_GB300_H */
