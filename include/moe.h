/*
 * moe.h -- C ABI of expert routing, dispatch planning and combination, same library as mxfp8.h, whose
 * conventions hold here (the caller's buffers, status codes, stream order, no allocation, nothing read on
 * the host).  Row-major throughout; types are those of mxfp4.h.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#include "mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_MAX_TOPK 32

typedef enum {
    MOE_SOFTMAX = 0, /* p_e = exp(l_e - max l) / sum exp(l - max l); a row of -inf only: all p = 0 */
    MOE_SIGMOID = 1  /* p_e = 1 / (1 + exp(-l_e)) */
} moe_score_t;

/*
 * Options of moe_route.  Experts are chosen by a key: the logit itself without a bias (scores rise with
 * it), score + bias[e] with one.  With topk_groups < num_groups only the experts of the topk_groups best of
 * num_groups equal groups (consecutive experts) can be chosen; a group's rank is its largest key, or with a
 * bias the sum of its two largest.  Ties go to the lower index; a NaN ranks below every number.  The bias
 * enters the choice alone.  Weights are scale * p, or scale * p / (sum of the chosen p) with renormalize
 * (all 0 if that sum is 0).
 */
typedef struct moe_route_config {
    int score;         /* moe_score_t */
    int top_k;         /* 1 .. min(MOE_MAX_TOPK, experts that can be chosen) */
    int num_groups;    /* >= 1, divides E */
    int topk_groups;   /* 1 .. num_groups */
    int renormalize;   /* 0 or 1 */
    float scale;
    const float *bias; /* device fp32 [E] or NULL */
    int reserved[4];   /* must be 0 */
} moe_route_config_t;

/*
 * Route T tokens over E experts (1 <= E <= MXFP8_MAX_GROUPS): indices int32 [T, top_k] by falling key,
 * weights fp32 [T, top_k].  logits [T, E], type MXFP4_BF16 or MXFP4_F32, row pitch ld >= E.
 * The sum of the softmax is formed in one fixed order: halves of the row padded with zeros to 512 experts
 * are added until one value is left (p_e and p_(e + 256), then e and e + 128, ...).
 */
mxfp8_status_t moe_route(const void *logits, int type, int64_t T, int64_t E, int64_t ld, const moe_route_config_t *cfg,
                         int32_t *indices, float *weights, void *stream);

/*
 * The gradient of moe_route's weights: dlogits [T, E] (type and row pitch E) from dweights fp32 [T, top_k]
 * and the indices that moe_route chose (constants, like the bias).  Uses score, top_k, renormalize and
 * scale of cfg.  An index outside [0, E) is left out.  With d_j = scale * dweights_j, and with renormalize
 * d_j <- (d_j - sum_i d_i p_i / S) / S, S = sum of the chosen p (0 if S is 0):
 *     softmax:  dl_e = p_e * (sum_{j: idx_j = e} d_j - sum_j d_j p_j);   sigmoid:  dl_e = d_e p_e (1 - p_e).
 */
mxfp8_status_t moe_route_backward(const void *logits, int type, int64_t T, int64_t E, int64_t ld,
                                  const moe_route_config_t *cfg, const int32_t *indices, const float *dweights,
                                  void *dlogits, void *stream);

/* Device workspace of moe_plan for n = T * top_k choices over E experts (4-byte aligned). */
size_t moe_plan_workspace_bytes(int64_t n, int64_t E);

/*
 * Sort the n = T * k choices `indices` by expert, keeping their order within an expert (deterministic):
 *   offsets  int64 [E + 1]: expert e's rows are [offsets[e], offsets[e+1])
 *   slots    int32 [n]: the row of each choice.  A choice outside [0, E) is dropped: it gets -2 - r for one
 *            of the rows r >= offsets[E] that are left over
 *   tokens   int32 [n]: the token (choice / k) of each row; -1 for the rows left over
 * n < 2^31.  workspace: moe_plan_workspace_bytes(n, E) bytes.
 */
mxfp8_status_t moe_plan(const int32_t *indices, int64_t n, int k, int64_t E, int64_t *offsets, int32_t *slots,
                        int32_t *tokens, void *workspace, void *stream);

/*
 * out[t, :] = sum_j weights[t, j] * y[slots[t, j], :] for j = 0 .. k-1 in that order, in fp32, rounded once to
 * bf16.  y bf16 [R, H], H a multiple of 8; slots outside [0, R) add nothing; weights NULL = all 1 (the
 * gradient of the gather that moe_plan's tokens describe).  1 <= k <= MOE_MAX_TOPK.
 */
mxfp8_status_t moe_combine(const void *y, int64_t R, int64_t H, const int32_t *slots, const float *weights, int64_t T,
                           int k, void *out, void *stream);

/*
 * Its gradient: dy[slots[t, j], :] = weights[t, j] * dout[t, :] (bf16 [R, H]) and dweights[t, j] = sum_h
 * dout[t, h] * y[slots[t, j], h] (fp32, fixed order; 0 for a slot outside [0, R)).  The slots name distinct
 * rows; a slot of -2 - r sets row r of dy to zeros, so that moe_plan's slots write every row of their n; rows
 * that no slot names are left as they are.  Either output may be NULL, and y without dweights.
 */
mxfp8_status_t moe_combine_backward(const void *dout, const void *y, int64_t R, int64_t H, const int32_t *slots,
                                    const float *weights, int64_t T, int k, void *dy, float *dweights, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_H */
