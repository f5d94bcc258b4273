/*
 * mccb_ssm.h -- the operators around the causal depthwise convolution in a selective state space
 * block, on AMD Instinct MI355X (gfx950): the convolution with its bias, activation and carried
 * rows, the selective scan, and the matrix product with its epilogue; each with its backward, and
 * the first two with their single-token form.
 *
 * Conventions are those of mccb.h: raw device pointers, caller-owned buffers, a
 * ..._get_workspace_size call (host only, no HIP call) before each call that needs a workspace,
 * status codes, work enqueued on `stream` (a hipStream_t; NULL = the default stream) without
 * waiting. All checks run on the host before any HIP call, and on an error nothing is enqueued:
 * NULL pointers (MCCB_ERR_PARAM_NULLPTR), dtype, activation, strides, alignment, overlap and
 * workspace (MCCB_ERR_PARAM_INVALID), sizes (MCCB_ERR_SHAPE); MCCB_ERR_RUNTIME reports a launch
 * that the HIP runtime refused, before which a call's earlier kernels may have been enqueued.
 * Nothing is allocated and nothing is kept between calls, so every call can be recorded into a HIP
 * graph. Results are the same bits on every call with the same inputs.
 *
 * Data tensors are time-major, [S,B,...], as in mccb.h, and are read through element strides
 * (>= 0; 0 repeats). Element strides are in the tensor's own elements. Outputs are contiguous, are
 * overwritten, and overlap no other buffer. 16-bit buffers are 2-byte, 32-bit ones 4-byte aligned,
 * workspaces and `saved` 16-byte.
 *
 * lengths: optional int64 [B] on the device, clamped to [0, S]; NULL = all S. Rows at or past a
 * sequence's length are not computed with, whatever they hold (also infinities and NaN): outputs
 * and gradients there are zero, and states are those after the last row before it. A length of
 * zero hands the initial state on.
 */
#ifndef MCCB_SSM_H
#define MCCB_SSM_H

#include <stdint.h>

#include "mccb.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations. gelu is the tanh form: v/2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))). */
typedef enum {
    MCCB_ACT_NONE = 0,
    MCCB_ACT_RELU = 1,
    MCCB_ACT_SILU = 2,
    MCCB_ACT_GELU = 3,
    MCCB_ACT_SOFTPLUS = 4
} mccb_act_t;

/* ------------------------------------------------------------------------------------------------
 * Causal depthwise convolution with bias, activation and carried rows.
 *
 *   y[t,b,h] = act(bias[h] + sum_{k<W} weight[k,h] x[t-W+1+k,b,h]),
 *
 * rows before the first taken from `state` (state[r] is row r-W+1), or zero without one. Products
 * of two 16-bit values are exact in fp32; the sum, the activation and the gradients are fp32, rounded
 * once. gradWeight and gradBias add strips of up to 64 rows, and four of those, in fp32 and go on in
 * fp64 over rows and batches (strips grow from S = 65535 * 64 on).
 *
 * B in [1, 65535], S in [0, 2^31), H in [1, 2^24], B H < 2^31, W in 1..4; activation none or silu.
 * -----------------------------------------------------------------------------------------------*/
typedef struct {
    int64_t S, B, H, W;
    int32_t dtype, activation;
    const void *x;           /* [S,B,H] */
    int64_t x_stride[3];     /* along S, B, H */
    const void *weight;      /* [W,H] contiguous */
    const void *bias;        /* [H] or NULL */
    const int64_t *lengths;  /* [B] or NULL */
    const void *state;       /* [W-1,B,H] contiguous: the rows before the first; NULL = zeros */
} mccb_conv_t;

/* y [S,B,H]; final_state [W-1,B,H] or NULL: the last W-1 rows before each sequence's length (from
 * `state` where the sequence is shorter). No workspace. */
int mccb_conv_act_forward(const mccb_conv_t *args, void *y, void *final_state, void *stream);

/* The gradients, from the same arguments as the forward and
 *   gradY [S,B,H] (strides gy_stride), gradFinalState [W-1,B,H] contiguous or NULL.
 * gradX [S,B,H] and gradWeight [W,H] are required, gradBias [H] and gradState [W-1,B,H] optional.
 * The pre-activation is computed again from x. */
int mccb_conv_act_backward_get_workspace_size(const mccb_conv_t *args, uint64_t *workspace_size);
int mccb_conv_act_backward(const mccb_conv_t *args, const void *gradY, const int64_t *gy_stride,
                           const void *gradFinalState, void *gradX, void *gradWeight,
                           void *gradBias, void *gradState, void *workspace,
                           uint64_t workspace_size, void *stream);

/* One token: x and y [B,H] (args->S = 1, x_stride[0] unused); `state` [W-1,B,H] is read and then
 * shifted up by one row in place. args->state and args->lengths are NULL. */
int mccb_conv_act_step(const mccb_conv_t *args, void *state, void *y, void *stream);

/* ------------------------------------------------------------------------------------------------
 * Selective state space scan. For every channel h of group g = h / (H/G) and state n < N:
 *
 *   d[t]   = softplus(dt[t,b,h] + dt_bias[h])        (without softplus: the sum itself)
 *   s[t,n] = exp(d[t] A[n,h]) s[t-1,n] + d[t] Bm[t,b,g,n] x[t,b,h]
 *   y[t]   = sum_n Cm[t,b,g,n] s[t,n] + D[h] x[t]
 *   out[t] = y[t] silu(z[t])                         (without z: y[t])
 *
 * x, dt, z, out, Bm and Cm have the dtype, A, D, dt_bias and the states are fp32; everything is
 * computed in fp32 and rounded once. Gradients' sums: gradB and gradC add 64 channels in fp32 and such
 * blocks in fp64; gradA adds 16 rows in fp32, gradD and gradDtBias every 16th row of up to 512 and
 * then those sums, and all go on in fp64 over rows (gradA), chunks and batches. Every order is fixed.
 *
 * B in [1, 65535], S in [0, 2^31), H in [1, 2^24], B H < 2^31, G in [1, 2^22] and a divisor of H, N in
 * 1..32.
 * -----------------------------------------------------------------------------------------------*/
typedef struct {
    int64_t S, B, H, N, G;
    int32_t dtype, softplus;  /* softplus: nonzero = applied */
    const void *x, *dt;       /* [S,B,H] */
    const void *z;            /* [S,B,H] or NULL */
    const void *Bm, *Cm;      /* [S,B,G,N] */
    int64_t x_stride[3], dt_stride[3], z_stride[3]; /* along S, B, H */
    int64_t b_stride[4], c_stride[4];               /* along S, B, G, N */
    const float *A;           /* [N,H] contiguous */
    const float *D;           /* [H] or NULL (zero) */
    const float *dt_bias;     /* [H] or NULL (zero) */
    const int64_t *lengths;   /* [B] or NULL */
    const float *state;       /* [B,N,H] contiguous, the state before the first row; NULL = zeros */
} mccb_scan_t;

/* out [S,B,H]; final_state [B,N,H] or NULL; saved: NULL, or mccb_scan_saved_size bytes that the
 * backward reads (the state before every 16th row). */
int mccb_scan_saved_size(const mccb_scan_t *args, uint64_t *bytes);
int mccb_scan_forward_get_workspace_size(const mccb_scan_t *args, uint64_t *workspace_size);
int mccb_scan_forward(const mccb_scan_t *args, void *out, float *final_state, void *saved,
                      void *workspace, uint64_t workspace_size, void *stream);

/* Gradients. gradOut has strides gout_stride; gradFinalState may be NULL (zero). The [S,B,H] and
 * [S,B,G,N] outputs are contiguous and required, except gradZ (required with z, else NULL); gradA is
 * required, gradD, gradDtBias and gradState are optional. */
typedef struct {
    const void *gradOut;          /* [S,B,H] */
    int64_t gout_stride[3];       /* along S, B, H */
    const float *gradFinalState;  /* [B,N,H] or NULL */
    void *gradX, *gradDt, *gradZ; /* [S,B,H] */
    void *gradB, *gradC;          /* [S,B,G,N] */
    float *gradA;                 /* [N,H] */
    float *gradD, *gradDtBias;    /* [H] or NULL */
    float *gradState;             /* [B,N,H] or NULL */
} mccb_scan_grads_t;

int mccb_scan_backward_get_workspace_size(const mccb_scan_t *args, uint64_t *workspace_size);
int mccb_scan_backward(const mccb_scan_t *args, const mccb_scan_grads_t *grads, const void *saved,
                       void *workspace, uint64_t workspace_size, void *stream);

/* One token: x, dt, z and out [B,H], Bm and Cm [B,G,N] (args->S = 1, the strides along S unused);
 * `state` [B,N,H] is updated in place. args->state and args->lengths are NULL. */
int mccb_scan_step(const mccb_scan_t *args, float *state, void *out, void *stream);

/* ------------------------------------------------------------------------------------------------
 * Matrix product with bias, activation and residual in its epilogue:
 *
 *   pre = x weight^T + bias,  out = act(pre) + residual
 *
 * x [M,K] and weight [N,K] have contiguous rows x_ld and weight_ld elements apart; bias [N],
 * residual [M,N] (rows residual_ld apart) and everything else have the same dtype. Products are
 * accumulated in fp32; bias, activation and residual are applied in fp32 and the result is rounded
 * once.
 *
 * M in [0, 2^22 - 64], N and K in [1, 2^22 - 64].
 * -----------------------------------------------------------------------------------------------*/
typedef struct {
    int64_t M, K, N;
    int32_t dtype, activation;
    const void *x;      /* [M,K] */
    const void *weight; /* [N,K] */
    const void *bias;   /* [N] or NULL */
    int64_t x_ld, weight_ld;
    int32_t pre_fp32;   /* nonzero: pre is fp32, else of the dtype */
} mccb_linear_t;

/* out [M,N] contiguous; pre [M,N] contiguous or NULL: the pre-activation, for the backward;
 * residual may be NULL. */
int mccb_linear_forward_get_workspace_size(const mccb_linear_t *args, uint64_t *workspace_size);
int mccb_linear_forward(const mccb_linear_t *args, const void *residual, int64_t residual_ld,
                        void *out, void *pre, void *workspace, uint64_t workspace_size,
                        void *stream);

/* With g = gradOut act'(pre): gradX = g weight [M,K], gradWeight = g^T x [N,K], gradBias = column
 * sums [N]. Each may be NULL and is then not computed; gradient of the residual is gradOut itself.
 * pre is needed unless the activation is none. gradOut's rows are gout_ld elements apart.
 * Two roundings to the dtype lie between these gradients and the exact ones, besides their own:
 *   - g's, since the matrix instructions take 16-bit operands (gradBias sums it before);
 *   - pre's, unless it is kept in fp32: act' is then taken up to half a step of pre away. */
int mccb_linear_backward_get_workspace_size(const mccb_linear_t *args, uint64_t *workspace_size);
int mccb_linear_backward(const mccb_linear_t *args, const void *gradOut, int64_t gout_ld,
                         const void *pre, void *gradX, void *gradWeight, void *gradBias,
                         void *workspace, uint64_t workspace_size, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MCCB_SSM_H */
