/*
 * pdssm_layers.h -- C ABI of the operators that stand beside the PD-SSM scan
 * in a sequence layer, on MI355X (gfx950): the gated delta rule and the norm
 * of queries and keys with the rotation by position.  Same library
 * (libpdssm.so), status codes and pdssm_strerror as pdssm.h.
 *
 * The gated delta rule.  Every value head h of every sequence b holds a state
 * S[Dk,Dv].  With the query and key head hk = h / (Hv / Hk), and S before the
 * first step s0 (zero when s0 is NULL), step t does
 *     S   <- exp(g[b,h,t]) S
 *     u    = beta[b,h,t] (v[b,h,t,:] - S^T k[b,hk,t,:])
 *     S   <- S + k[b,hk,t,:] u^T
 *     o[b,h,t,:] = scale S^T q[b,hk,t,:]
 * and s_final is S after the last step.  g is a log decay of any sign; one
 * whose e^g rounds to zero in fp32 (g below -104, -inf and the lowest finite
 * value among them) empties the state before the step: a new document begins.
 *
 * The norm with rotation.  For every head vector x of q and k (D values):
 *     y = x / sqrt(mean(x^2) + eps) * w       (RMS), or
 *     y = x / sqrt(sum(x^2) + eps) * w        (unit length, PDSSM_NORM_L2)
 * (w = 1 when NULL), then the first R dimensions turn in pairs by the angles
 * of the token's position p, c = cos[p,i] and s = sin[p,i] for i < R/2:
 *     (y[a], y[b]) <- (c y[a] - s y[b], s y[a] + c y[b])
 * with (a, b) = (i, i + R/2), or (2i, 2i + 1) with PDSSM_ROPE_PAIRS.
 *
 * Types: q, k, v, o, do and their gradients are bf16 with PDSSM_DATA_BF16,
 * else fp32.  Gates, states, weights, tables, and their gradients are fp32.
 * Arithmetic is fp32 or its equal (a product of fp32 values on the matrix
 * cores is taken as the sum of bf16 parts that together hold all 24 bits),
 * with one rounding to nearest even into a bf16 output.  Results are bitwise
 * reproducible.
 * A NaN or an infinity among the inputs of a step of pdssm_delta_fwd spoils
 * its heads' outputs from that step on and their state (in v, its column's
 * alone; in q, that step's outputs alone), and no output before; in
 * pdssm_delta_bwd it may spoil all gradients of its sequence.
 *
 * Layouts: device pointers.  q, k, v, o, g, beta and the like are indexed
 * [B,H,L(,D)] with the last dimension contiguous and the strides of the
 * first three, in elements, in the pdssm_strides of each; a NULL list means
 * contiguous [B,H,L(,D)]; for the delta rule the stride along L is in
 * [0, 2^23).  Rows need the alignment of their element only
 * (rows that all begin on 16 bytes are read faster).  States are contiguous
 * [B,Hv,Dk,Dv], 16-byte aligned.  Outputs overlap neither inputs nor each
 * other, except where said.
 *
 * The delta rule reads rows fastest whose head size is a multiple of 8 values
 * and that begin on 16 bytes, without overlapping.
 *
 * Ownership, execution and errors as in pdssm.h: the caller owns every buffer
 * and the workspace, which may hold anything on entry; the library allocates
 * nothing; every call is asynchronous on `stream`, and two calls in flight
 * need two workspaces.  Errors are found on the host before any HIP call
 * except PDSSM_ERR_HIP.
 */
#ifndef PDSSM_LAYERS_H
#define PDSSM_LAYERS_H

#include "pdssm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PDSSM_DATA_BF16 0x1u  /* q, k, v, o and their gradients are bf16 (else fp32) */
#define PDSSM_NORM_L2 0x2u    /* qk_norm_rope: unit length instead of RMS */
#define PDSSM_ROPE_PAIRS 0x4u /* qk_norm_rope: adjacent pairs (2i, 2i+1) instead of (i, i+R/2) */

/* Elements between neighbours along each of the first three dimensions. */
typedef struct {
    int64_t b, h, l;
} pdssm_strides;

/*
 * The gated delta rule over whole sequences (see above).
 *   q, k      [B,Hk,L,Dk]     v, o  [B,Hv,L,Dv]     g, beta  fp32 [B,Hv,L]
 *   s0        fp32 [B,Hv,Dk,Dv], or NULL for zero
 *   s_final   fp32 [B,Hv,Dk,Dv], or NULL when not wanted; may be s0
 *   strides   of q, k, v, g, beta, o, in this order, or NULL
 *   workspace pdssm_delta_workspace_bytes bytes, 16-byte aligned
 * Hv a multiple of Hk; Dk and Dv in [1,128]; flags: PDSSM_DATA_BF16.
 * B or Hv may be 0: nothing is read or written.  With L = 0, s_final = s0.
 */
int pdssm_delta_fwd(const void *q, const void *k, const void *v, const float *g,
                    const float *beta, const float *s0, void *o, float *s_final, int64_t B,
                    int64_t Hk, int64_t Hv, int64_t L, int32_t Dk, int32_t Dv, float scale,
                    uint32_t flags, const pdssm_strides *strides, void *workspace,
                    size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of pdssm_delta_fwd: 22 KB for every 64 steps of a value
 * head, and for long sequences of few heads (cut into at most about 1.5 times
 * the root of L / 64 segments) some states for each segment; 0 when the
 * arguments are invalid. */
size_t pdssm_delta_workspace_bytes(int64_t B, int64_t Hk, int64_t Hv, int64_t L, int32_t Dk,
                                   int32_t Dv, uint32_t flags);

/*
 * Gradients of pdssm_delta_fwd (reverse mode) from its inputs: the states
 * are made again from s0, nothing of the forward is kept.
 *   q, k, v, g, beta, s0   the forward's inputs
 *   d_o       [B,Hv,L,Dv], the gradient of o
 *   ds_final  fp32 [B,Hv,Dk,Dv], the gradient of s_final, or NULL for zero
 *   dq, dk    [B,Hk,L,Dk], each the sum over the value heads of its group
 *   dv        [B,Hv,L,Dv]
 *   dg, dbeta fp32 [B,Hv,L]
 *   ds0       fp32 [B,Hv,Dk,Dv], or NULL when not wanted; may be ds_final
 *   strides   of q, k, v, g, beta, d_o, dq, dk, dv, dg, dbeta, or NULL
 *   workspace pdssm_delta_bwd_workspace_bytes bytes, 16-byte aligned
 * Sizes, flags and empty shapes as pdssm_delta_fwd; with L = 0,
 * ds0 = ds_final (or zero).  dg is 0 where g empties the state (below
 * -104), and for the first step without s0.
 */
int pdssm_delta_bwd(const void *q, const void *k, const void *v, const float *g,
                    const float *beta, const float *s0, const void *d_o, const float *ds_final,
                    void *dq, void *dk, void *dv, float *dg, float *dbeta, float *ds0, int64_t B,
                    int64_t Hk, int64_t Hv, int64_t L, int32_t Dk, int32_t Dv, float scale,
                    uint32_t flags, const pdssm_strides *strides, void *workspace,
                    size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of pdssm_delta_bwd: for every 64 steps of a value head, the
 * state and its gradient (8 Dk Dv bytes), two vectors of Dv for each step and
 * 32 KB, and states for each segment as pdssm_delta_fwd; 0 when the arguments
 * are invalid. */
size_t pdssm_delta_bwd_workspace_bytes(int64_t B, int64_t Hk, int64_t Hv, int64_t L, int32_t Dk,
                                       int32_t Dv, uint32_t flags);

/*
 * One step of the gated delta rule for every sequence (decoding).
 *   q, k  [B,Hk,Dk]    v, o  [B,Hv,Dv]    g, beta  fp32 [B,Hv]
 *   s, s_out  fp32 [B,Hv,Dk,Dv]: the state before and after the step; s_out
 *         may be s (in place)
 *   strides  of q, k, v, g, beta, o (l is not used), or NULL
 * Sizes and flags as pdssm_delta_fwd.  B or Hv may be 0.
 */
int pdssm_delta_step(const void *q, const void *k, const void *v, const float *g,
                     const float *beta, const float *s, void *o, float *s_out, int64_t B,
                     int64_t Hk, int64_t Hv, int32_t Dk, int32_t Dv, float scale, uint32_t flags,
                     const pdssm_strides *strides, hipStream_t stream);

/*
 * Norm of every query and key head with the rotation by position (see above).
 *   q, q_out  [B,Hq,L,D]    k, k_out  [B,Hk,L,D]   (an output may be its input)
 *   wq, wk    fp32 [D], or NULL for 1
 *   cos, sin  fp32 [P,R/2] (R = 0: not read), 16-byte aligned when R is a
 *             multiple of 16
 *   pos       int32 [B,L] positions, clamped to [0,P), or NULL for pos = l
 *   strides   of q, k, q_out, k_out, or NULL
 * D in [1,256]; R even, in [0,D]; P >= 1 when R > 0; Hq and Hk up to 32768,
 * B*L*(Hq+Hk) below 2^31; any of B, Hq, Hk, L may
 * be 0.  flags: PDSSM_DATA_BF16, PDSSM_NORM_L2, PDSSM_ROPE_PAIRS.
 */
int pdssm_qk_norm_rope_fwd(const void *q, const void *k, const float *wq, const float *wk,
                           const float *cos, const float *sin, const int32_t *pos, void *q_out,
                           void *k_out, int64_t B, int64_t Hq, int64_t Hk, int64_t L, int32_t D,
                           int32_t R, int64_t P, float eps, uint32_t flags,
                           const pdssm_strides *strides, hipStream_t stream);

/*
 * Gradients of pdssm_qk_norm_rope_fwd from its inputs.
 *   dq_out, dk_out  gradients of the outputs, [B,Hq,L,D] and [B,Hk,L,D]
 *   dq, dk          gradients of the inputs (each may be its output gradient)
 *   dwq, dwk        fp32 [D] gradients of the weights, or NULL when not
 *                   wanted (a weight of NULL counts as ones)
 *   strides         of q, k, dq_out, dk_out, dq, dk, or NULL
 *   workspace       pdssm_qk_norm_rope_bwd_workspace_bytes bytes, 16-byte
 *                   aligned; NULL when neither dwq nor dwk is wanted
 * With no rows, dwq and dwk are zero.
 */
int pdssm_qk_norm_rope_bwd(const void *q, const void *k, const float *wq, const float *wk,
                           const float *cos, const float *sin, const int32_t *pos,
                           const void *dq_out, const void *dk_out, void *dq, void *dk, float *dwq,
                           float *dwk, int64_t B, int64_t Hq, int64_t Hk, int64_t L, int32_t D,
                           int32_t R, int64_t P, float eps, uint32_t flags,
                           const pdssm_strides *strides, void *workspace, size_t workspace_bytes,
                           hipStream_t stream);

/* Workspace bytes of pdssm_qk_norm_rope_bwd with a weight gradient (a few MB
 * at most, whatever the sizes); 0 when the arguments are invalid. */
size_t pdssm_qk_norm_rope_bwd_workspace_bytes(int64_t B, int64_t Hq, int64_t Hk, int64_t L,
                                              int32_t D);

#ifdef __cplusplus
}
#endif

#endif /* PDSSM_LAYERS_H */
