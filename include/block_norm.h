/*
 * block_norm.h -- C ABI of the norms around a block (a layer's attention or experts), fused with its gate and residual
 * scale, and of their gradients; same library as mxfp8.h, whose conventions hold here (the caller's buffers, status
 * codes, stream order, no allocation, nothing read on the host).
 *
 * A block's output y joins the residual stream h [T, H], and the next block reads the stream's norm:
 *     r1 = 1 / sqrt(mean(y^2) + eps)   u = y r1 w_post      (u = y without w_post)
 *     h' = scale h + gate u            rounded to h's type: the stream as it is kept
 *     r2 = 1 / sqrt(mean(h'^2) + eps)  x = h' r2 w_pre      of the rounded h', rounded to bf16
 * means over a row, in fp32.  gate is a factor per channel or per token.
 */
#ifndef BLOCK_NORM_GB300_H
#define BLOCK_NORM_GB300_H

#include <stddef.h>
#include <stdint.h>

#include "mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BLOCK_NORM_MAX_H 16384

typedef enum {
    BLOCK_GATE_NONE = 0,
    BLOCK_GATE_CHANNEL = 1, /* fp32 [H] */
    BLOCK_GATE_TOKEN = 2    /* fp32 [T] */
} block_gate_t;

typedef struct block_norm_config {
    int y_type;               /* MXFP4_BF16 or MXFP4_F32 */
    int h_type;               /* of the stream, in and out, and of its gradients */
    int gate_kind;            /* block_gate_t */
    float scale;
    float eps;
    const float *pre_weight;  /* device fp32 [H], or NULL: no norm of the stream, no x */
    const float *post_weight; /* device fp32 [H], or NULL: no norm of y */
    const float *gate;        /* device fp32, NULL with BLOCK_GATE_NONE */
    int reserved[4];          /* must be 0 */
} block_norm_config_t;

/*
 * Forward.  y [T, H] (pitch ldy) or NULL (no block: h' = scale h; then no post_weight and no gate), h [T, H] (pitch ldh);
 * h_out [T, H] of h's type, or NULL; x [T, H] bf16, NULL without pre_weight.  Outputs have pitch H; h_out may be h itself
 * where ldh is H.  H and pitches multiples of 8, H <= BLOCK_NORM_MAX_H, T < 2^31; all row pointers 16-byte aligned,
 * weights and gates 16-byte (a gate per token 4-byte).
 * MXFP8_ERR_FORMAT (types, gate_kind, reserved), _SHAPE, _NULL, _ALIGN, _DEVICE, _LAUNCH.
 */
mxfp8_status_t block_norm(const block_norm_config_t *cfg, int64_t T, int64_t H, const void *y, int64_t ldy, const void *h,
                          int64_t ldh, void *h_out, void *x, void *stream);

/* Device workspace of block_norm_backward, 16-byte aligned. */
size_t block_norm_backward_workspace_bytes(int64_t T, int64_t H);

/*
 * Gradients, from those of h' and x (dh_out of h's type, dx bf16; either may be NULL: none; dx only with pre_weight), y
 * and the stream h_out that the forward pass left.  With g the whole gradient of h',
 *     t = dx w_pre, n2 = h' r2:   g = dh_out + r2 (t - n2 mean(t n2)),  dpre = sum over tokens of dx n2,  dh = scale g
 *     n1 = y r1, b = gate g w_post:  dy = r1 (b - n1 mean(b n1)),  dpost = sum over tokens of gate g n1   (dy = gate g
 *     without post_weight),  dgate = sum of g u over tokens (per channel) or over the row (per token)
 * sums in fp32 in a fixed order.  dh [T, H] of h's type and dy of y's, pitch H; dpre, dpost [H] and dgate [H] or [T] fp32.
 * Any output may be NULL.  y may be NULL where neither post_weight nor a gate's gradient needs it.
 * MXFP8_ERR_WORKSPACE without a workspace (needed when T and H are not 0).
 */
mxfp8_status_t block_norm_backward(const block_norm_config_t *cfg, int64_t T, int64_t H, const void *dh_out, int64_t lddh,
                                   const void *dx, int64_t lddx, const void *y, int64_t ldy, const void *h_out,
                                   int64_t ldh, void *dh, void *dy, float *dpre, float *dpost, float *dgate,
                                   void *workspace, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* BLOCK_NORM_GB300_H */
