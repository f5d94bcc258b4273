/*
 * mccb_delta.h -- the gated delta rule, and the norms before and after a block, on AMD Instinct MI355X
 * (gfx950): what a block around the causal depthwise convolution runs in place of the selective scan of
 * mccb_ssm.h, and what stands around such a block; each with its backward, and the delta rule with its
 * single-token form.
 *
 * Conventions are those of mccb_ssm.h: raw device pointers, caller-owned buffers, a
 * ..._get_workspace_size call (host only, no HIP call) before each call that needs a workspace, status
 * codes, work enqueued on `stream` without waiting, all checks on the host before any HIP call, nothing
 * allocated and nothing kept between calls, the same bits on every call with the same inputs. Outputs are
 * contiguous, are overwritten, and overlap no other buffer. 16-bit buffers are 2-byte, 32-bit ones
 * 4-byte aligned, workspaces and `saved` 16-byte.
 */
#ifndef MCCB_DELTA_H
#define MCCB_DELTA_H

#include <stdint.h>

#include "mccb.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------------------
 * Norms before and after a block, over rows of H values:
 *
 *   prenorm   sum = residual + scale x,  out = sum / sqrt(mean(sum^2) + eps) weight
 *   postnorm  out = residual + scale (x / sqrt(mean(x^2) + eps) weight silu(z))
 *
 * prenorm's mean is over the row; postnorm's over each of `groups` equal parts of it, with a weight of
 * its own for every value, or (weight_shared) one of H/groups values for all groups. residual, scale [H]
 * and z may be NULL: then their factor or term is left out. Everything has the dtype, is computed in fp32
 * and rounded once; prenorm's norm is of the sum before its rounding. Gradients of weight and scale add
 * a block's rows in fp32 (8 to R/1024 of them, and one block's at most where there are fewer) and go on in
 * fp64. Rows are contiguous and x_ld, residual_ld, z_ld elements apart; results are contiguous.
 *
 * R in [0, 2^31), H in [1, 2^24], groups in [1, 65535] and a divisor of H, H/groups up to 16384, eps
 * positive. prenorm has groups = 1 and no z.
 * -----------------------------------------------------------------------------------------------*/
typedef struct {
    int64_t R, H, groups;
    int32_t dtype, weight_shared;
    float eps;
    const void *x, *weight, *residual, *scale, *z;
    int64_t x_ld, residual_ld, z_ld;
} mccb_norm_t;

/* out [R,H]; sum [R,H] or NULL. No workspace. */
int mccb_prenorm_forward(const mccb_norm_t *args, void *out, void *sum, void *stream);
int mccb_postnorm_forward(const mccb_norm_t *args, void *out, void *stream);

/* Gradients, from the same arguments and gradOut [R,H] (rows gout_ld apart); the normalized values are
 * computed again. gradSum [R,H], the gradient that reaches prenorm's sum from elsewhere, may be NULL.
 * gradX and gradWeight are required, gradScale and gradZ with scale and z (else NULL). prenorm's
 * gradResidual may be NULL, and is gradX itself where there is no scale; postnorm's is gradOut. */
int mccb_prenorm_backward_get_workspace_size(const mccb_norm_t *args, uint64_t *workspace_size);
int mccb_prenorm_backward(const mccb_norm_t *args, const void *gradOut, int64_t gout_ld,
                          const void *gradSum, int64_t gsum_ld, void *gradX, void *gradResidual,
                          void *gradWeight, void *gradScale, void *workspace, uint64_t workspace_size,
                          void *stream);
int mccb_postnorm_backward_get_workspace_size(const mccb_norm_t *args, uint64_t *workspace_size);
int mccb_postnorm_backward(const mccb_norm_t *args, const void *gradOut, int64_t gout_ld, void *gradX,
                           void *gradZ, void *gradWeight, void *gradScale, void *workspace,
                           uint64_t workspace_size, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MCCB_DELTA_H */
