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
 * Gated delta rule. For every value head h, of key head g = h / (H/G), a state S [K,V]:
 *
 *   d    = softplus(dt[t,b,h] + dt_bias[h])       (without softplus: the sum itself)
 *   a    = exp(A[h] d),  beta = sigmoid(b[t,b,h])
 *   kn   = k / sqrt(sum(k^2) + 1e-6),  qn = q / sqrt(sum(q^2) + 1e-6)     (without normalize: k and q)
 *   u    = beta (v[t,b,h] - a S^T kn)
 *   S    = a S + kn u^T
 *   out  = scale S^T qn
 *
 * q, k [S,B,G,K], v and out [S,B,H,V], dt and b [S,B,H] have the dtype; A, dt_bias [H] and the states are
 * fp32. Rows of q, k and v are contiguous; the other axes have element strides (>= 0; 0 repeats). Gates and
 * decays are computed in fp32, sums of their logarithms in fp64. delta_step computes in fp32. The other
 * calls go by chunks of 64 rows, in products of two 16-bit terms for each operand and fp32 sums: what a
 * product takes of states, U and gradients has 22 bits next to the largest value of its column or row in the
 * chunk, fewer below 2^-18 of that, and nothing below 2^-40. A small row of k or q, or a row of zeros, takes
 * none from the others and loses none itself. Outputs and gradients are rounded once to 16 bits. Rates A are negative in ordinary use (decay); A d below -1e5
 * counts as -1e5, whose decay is 0.
 *
 * lengths: optional int64 [B] on the device, clamped to [0, S]; NULL = all S. Rows at or past a sequence's
 * length are not computed with, whatever they hold: outputs and gradients there are zero, and states are
 * those after the last row before it. A length of zero hands the initial state on. A live row that is not
 * finite makes NaN of what comes after it in its sequence, and of up to 63 rows before it (its chunk's).
 *
 * S in [0, 2^28), B H in [1, 65535], G a divisor of H, K in 1..128, V in 1..256, scale finite.
 * -----------------------------------------------------------------------------------------------*/
typedef struct {
    int64_t S, B, H, G, K, V;
    int32_t dtype, softplus, normalize;  /* softplus, normalize: nonzero = applied */
    float scale;
    const void *q, *k, *v, *dt, *b;
    int64_t q_stride[3], k_stride[3];    /* along S, B, G */
    int64_t v_stride[3], dt_stride[3], b_stride[3]; /* along S, B, H */
    const float *A;           /* [H] */
    const float *dt_bias;     /* [H] or NULL (zero) */
    const int64_t *lengths;   /* [B] or NULL */
    const float *state;       /* [B,H,K,V] contiguous, the state before the first row; NULL = zeros */
} mccb_delta_t;

/* out [S,B,H,V]; final_state [B,H,K,V] or NULL; saved: NULL, or mccb_delta_saved_size bytes that the
 * backward reads: for every 64 rows of a head the state before them and their U in fp32, K counted as 64 or
 * 128 and V in steps of 64 (at K = V = 128 and G = H 2.4 KB a row and head with the chunk's matrices; the
 * backward's workspace is another 1.5 KB). With saved no workspace is needed. */
int mccb_delta_saved_size(const mccb_delta_t *args, uint64_t *bytes);
int mccb_delta_forward_get_workspace_size(const mccb_delta_t *args, uint64_t *workspace_size);
int mccb_delta_forward(const mccb_delta_t *args, void *out, float *final_state, void *saved,
                       void *workspace, uint64_t workspace_size, void *stream);

/* Gradients. gradOut has strides gout_stride and contiguous rows; gradFinalState may be NULL (zero). Outputs
 * are contiguous and required, except gradDtBias and gradState. Gradients of q and k add the value heads
 * of a key head in fp32; gradA and gradDtBias add rows and chunks in fp64. Every order is fixed. */
typedef struct {
    const void *gradOut;           /* [S,B,H,V] */
    int64_t gout_stride[3];        /* along S, B, H */
    const float *gradFinalState;   /* [B,H,K,V] or NULL */
    void *gradQ, *gradK;           /* [S,B,G,K] */
    void *gradV;                   /* [S,B,H,V] */
    void *gradDt, *gradB;          /* [S,B,H] */
    float *gradA, *gradDtBias;     /* [H]; gradDtBias may be NULL */
    float *gradState;              /* [B,H,K,V] or NULL */
} mccb_delta_grads_t;

int mccb_delta_backward_get_workspace_size(const mccb_delta_t *args, uint64_t *workspace_size);
int mccb_delta_backward(const mccb_delta_t *args, const mccb_delta_grads_t *grads, const void *saved,
                        void *workspace, uint64_t workspace_size, void *stream);

/* One token: q, k [B,G,K], v and out [B,H,V], dt and b [B,H] (args->S = 1, the strides along S unused);
 * `state` [B,H,K,V] is updated in place. args->state and args->lengths are NULL. */
int mccb_delta_step(const mccb_delta_t *args, float *state, void *out, void *stream);

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
 * a block's rows in fp32 (about R groups/1024 of them, 4 at least, where R is as large) and go on in fp64.
 * Rows are contiguous and x_ld, residual_ld, z_ld elements apart; results are contiguous.
 *
 * R in [0, 2^31), H in [1, 2^24], groups in [1, 65535] and a divisor of H, H/groups up to 16384, eps
 * at least 2^-126. prenorm has groups = 1 and no z.
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
