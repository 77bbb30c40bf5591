/*
 * pdssm_block.h -- C ABI of further operators of a sequence layer's block, on
 * MI355X (gfx950): linear attention with decays, the layer norm with what
 * stands before it (dropout and the residual), and dropout.  Same library
 * (libpdssm.so), status codes and pdssm_strerror as pdssm.h; pdssm_strides and
 * PDSSM_DATA_BF16 as in pdssm_layers.h.
 *
 * Linear attention.  Every value head h of every sequence b holds a state
 * S[Dk,Dv].  With the query and key head hk = h / (Hv / Hk), and S before the
 * first step s0 (zero when s0 is NULL), step t does
 *     S   <- exp(g[b,h,t]) S + k[b,hk,t,:] v[b,h,t,:]^T
 *     o[b,h,t,:] = scale S^T q[b,hk,t,:]
 * and s_final is S after the last step.  g is a log decay of any sign, with any
 * strides (0 among them: a fixed decay for each head), or NULL for none; one
 * whose e^g rounds to zero in fp32 (g below -104, -inf and the lowest finite
 * value among them) empties the state before the step: a new document begins.
 * Where g is positive, states and results (before their scale too; for the gradient
 * of g the product of the norms of the state and its gradient) have to be numbers
 * that fp32 holds, e^g and the products of several need not (a state of zeros stays
 * zero); sequences whose positive gates add up to more than 60 in a run of 64 steps
 * are slower.
 *
 * The layer norm.  For every row of D values
 *     h = residual + dropout(x)                    (residual 0 when NULL)
 *     y = (h - mean(h)) / sqrt(var(h) + eps) * w + b
 * with var the mean of squares about the mean, w = 1 and b = 0 when NULL.  y is
 * of h before its rounding to the storage type.  A row's squares about its mean
 * have to add up to a number that fp32 holds (values up to 1e17 always do).
 *
 * Dropout.  With T = round(65536 p), a value is kept, and multiplied by
 * 65536 / (65536 - T), when its 16 random bits are T or more; the others become
 * zero, whatever they hold.  Value c of row r takes its bits from the block of
 * the Philox 4x32 generator with ten rounds (Salmon, Moraes, Dror and Shaw,
 * "Parallel random numbers: as easy as 1, 2, 3", 2011) whose counter is
 * (c / 8, r, low and high half of offset) and whose key is (low, high half of
 * seed): bits 16 (c % 2) .. 16 (c % 2) + 15 of word (c % 8) / 2.  No mask is
 * stored: the same seed and offset give the same one again, in any direction.
 * p is in [0, 1); T = 65536 counts as 65535.  seed and offset are arguments,
 * or, with `rng`, two values in device memory that the kernels read (a captured
 * graph then draws anew when they change between its replays).
 *
 * Types: q, k, v, o, x, residual, h, y and their gradients are bf16 with
 * PDSSM_DATA_BF16, else fp32.  Gates, states, weights and their gradients are
 * fp32.  Arithmetic is fp32 or its equal (a product of fp32 values on the
 * matrix cores is taken as the sum of bf16 parts that together hold all 24
 * bits), with one rounding to nearest even into a bf16 output.  Results are
 * bitwise reproducible.
 * A NaN or an infinity among the inputs of a step of pdssm_linear_fwd spoils
 * its heads' outputs from that step on and their state (in v its column of
 * both, in k its row of the state; in q its step's outputs alone); in
 * pdssm_linear_bwd it may spoil all gradients of its sequence.
 *
 * Layouts: device pointers.  Row tensors are indexed [B,H,L,D] (gates [B,H,L])
 * with the last dimension contiguous and the strides of the first three, in
 * elements, in the pdssm_strides of each; a NULL list means contiguous; for
 * linear attention the stride along L is in [0, 2^23).  Rows need the alignment
 * of their element only (rows that all begin on 16 bytes are read faster).
 * States are contiguous [B,Hv,Dk,Dv], 16-byte aligned.  Outputs overlap neither
 * inputs nor each other, except where said.
 *
 * Ownership, execution and errors as in pdssm.h: the caller owns every buffer
 * and the workspace, which may hold anything on entry; the library allocates
 * nothing; every call is asynchronous on `stream`, and two calls in flight
 * need two workspaces.  Errors are found on the host before any HIP call
 * except PDSSM_ERR_HIP.
 */
#ifndef PDSSM_BLOCK_H
#define PDSSM_BLOCK_H

#include "pdssm_layers.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PDSSM_NO_DG 0x2u    /* linear_bwd: dg is not wanted (dg may be NULL) */
#define PDSSM_DG_HEADS 0x4u /* linear_bwd: dg is [Hv], summed over sequences and steps */

/*
 * Linear attention over whole sequences (see above).
 *   q, k      [B,Hk,L,Dk]     v, o  [B,Hv,L,Dv]     g  fp32 [B,Hv,L] or NULL
 *   s0        fp32 [B,Hv,Dk,Dv], or NULL for zero
 *   s_final   fp32 [B,Hv,Dk,Dv], or NULL when not wanted; may be s0
 *   strides   of q, k, v, g, o, in this order, or NULL
 *   workspace pdssm_linear_workspace_bytes bytes, 16-byte aligned
 * Hv a multiple of Hk; Dk and Dv in [1,128]; flags: PDSSM_DATA_BF16.
 * B or Hv may be 0: nothing is read or written.  With L = 0, s_final = s0.
 */
int pdssm_linear_fwd(const void *q, const void *k, const void *v, const float *g, const float *s0,
                     void *o, float *s_final, int64_t B, int64_t Hk, int64_t Hv, int64_t L,
                     int32_t Dk, int32_t Dv, float scale, uint32_t flags,
                     const pdssm_strides *strides, void *workspace, size_t workspace_bytes,
                     hipStream_t stream);

/* Workspace bytes of pdssm_linear_fwd: 256, and for few heads, whose sequences
 * are cut into at most 256 segments together, a state for each segment; 0 when
 * the arguments are invalid. */
size_t pdssm_linear_workspace_bytes(int64_t B, int64_t Hk, int64_t Hv, int64_t L, int32_t Dk,
                                    int32_t Dv, uint32_t flags);

/*
 * Gradients of pdssm_linear_fwd (reverse mode) from its inputs: the states are
 * made again from s0, nothing of the forward is kept.
 *   q, k, v, g, s0   the forward's inputs
 *   d_o       [B,Hv,L,Dv], the gradient of o
 *   ds_final  fp32 [B,Hv,Dk,Dv], the gradient of s_final, or NULL for zero
 *   dq, dk    [B,Hk,L,Dk], each the sum over the value heads of its group
 *   dv        [B,Hv,L,Dv]
 *   dg        fp32 [B,Hv,L], with PDSSM_DG_HEADS fp32 [Hv] (stride h alone),
 *             the sum over sequences and steps; not written with PDSSM_NO_DG
 *   ds0       fp32 [B,Hv,Dk,Dv], or NULL when not wanted; may be ds_final
 *   strides   of q, k, v, g, d_o, dq, dk, dv, dg, or NULL
 *   workspace pdssm_linear_bwd_workspace_bytes bytes, 16-byte aligned
 * Sizes and empty shapes as pdssm_linear_fwd; with L = 0, ds0 = ds_final (or
 * zero), and dg [Hv] is zero (with B = 0 too).  flags: PDSSM_DATA_BF16 and one
 * of PDSSM_NO_DG, PDSSM_DG_HEADS.  dg is 0 where g empties the state (below
 * -104), and for the first step without s0.  The other gradients are the same
 * bits whether dg is wanted or not.
 */
int pdssm_linear_bwd(const void *q, const void *k, const void *v, const float *g, const float *s0,
                     const void *d_o, const float *ds_final, void *dq, void *dk, void *dv,
                     float *dg, float *ds0, int64_t B, int64_t Hk, int64_t Hv, int64_t L,
                     int32_t Dk, int32_t Dv, float scale, uint32_t flags,
                     const pdssm_strides *strides, void *workspace, size_t workspace_bytes,
                     hipStream_t stream);

/* Workspace bytes of pdssm_linear_bwd: with dg the state of every 64 steps of
 * a value head, with shared heads (Hv > Hk) dq and dk of every value head in
 * fp32, one state for each value head, and for few heads three for each segment
 * as pdssm_linear_fwd; 0 when the arguments are invalid. */
size_t pdssm_linear_bwd_workspace_bytes(int64_t B, int64_t Hk, int64_t Hv, int64_t L, int32_t Dk,
                                        int32_t Dv, uint32_t flags);

/*
 * One step of linear attention for every sequence (decoding).
 *   q, k  [B,Hk,Dk]    v, o  [B,Hv,Dv]    g  fp32 [B,Hv] or NULL
 *   s, s_out  fp32 [B,Hv,Dk,Dv]: the state before and after the step; s_out
 *         may be s (in place)
 *   strides  of q, k, v, g, o (l is not used), or NULL
 * Sizes and flags as pdssm_linear_fwd.  B or Hv may be 0.
 */
int pdssm_linear_step(const void *q, const void *k, const void *v, const float *g, const float *s,
                      void *o, float *s_out, int64_t B, int64_t Hk, int64_t Hv, int32_t Dk,
                      int32_t Dv, float scale, uint32_t flags, const pdssm_strides *strides,
                      hipStream_t stream);

/*
 * The layer norm of h = residual + dropout(x) (see above).
 *   x, residual, y, h  [B,H,L,D]; residual NULL for zero, h NULL when not
 *             wanted; y or h may be x or residual
 *   w, b      fp32 [D], or NULL for 1 and 0
 *   p, seed, offset, rng   the dropout (p = 0: none); rng NULL, or two values
 *             in device memory, 8-byte aligned, in place of seed and offset
 *   strides   of x, residual, y, h, or NULL
 * D in [1,16384]; B*H*L below 2^31; any of B, H, L may be 0.
 * flags: PDSSM_DATA_BF16.
 */
int pdssm_layer_norm_fwd(const void *x, const void *residual, const float *w, const float *b,
                         void *y, void *h, int64_t B, int64_t H, int64_t L, int32_t D, float eps,
                         double p, uint64_t seed, uint64_t offset, const uint64_t *rng,
                         uint32_t flags, const pdssm_strides *strides, hipStream_t stream);

/*
 * Gradients of pdssm_layer_norm_fwd from h (as stored) and dy, the gradient
 * of y.
 *   dh        the gradient that h has from elsewhere, or NULL for zero
 *   dr        the gradient of h (of the residual, and without dropout of x),
 *             or NULL when not wanted; may be dy, dh or h
 *   dx        the gradient of x, or NULL when not wanted; may be dy, dh or h,
 *             not dr
 *   dw, db    fp32 [D] gradients of w and b, or NULL when not wanted (a w of
 *             NULL counts as ones)
 *   strides   of h, dy, dh, dr, dx, or NULL
 *   workspace pdssm_layer_norm_bwd_workspace_bytes bytes, 16-byte aligned; NULL
 *             when neither dw nor db is wanted
 * With no rows, dw and db are zero.
 */
int pdssm_layer_norm_bwd(const void *h, const void *dy, const void *dh, const float *w, void *dr,
                         void *dx, float *dw, float *db, int64_t B, int64_t H, int64_t L,
                         int32_t D, float eps, double p, uint64_t seed, uint64_t offset,
                         const uint64_t *rng, uint32_t flags, const pdssm_strides *strides,
                         void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of pdssm_layer_norm_bwd with dw or db (512 rows of sums at
 * most); 0 when the arguments are invalid. */
size_t pdssm_layer_norm_bwd_workspace_bytes(int64_t B, int64_t H, int64_t L, int32_t D);

/*
 * y = residual + dropout(x) (see above); the gradient of x is dropout of y's
 * with the same seed and offset.
 *   x, residual, y  [B,H,L,D]; residual NULL for zero; y may be x or residual
 *   strides   of x, residual, y, or NULL
 * Sizes and flags as pdssm_layer_norm_fwd.
 */
int pdssm_dropout(const void *x, const void *residual, void *y, int64_t B, int64_t H, int64_t L,
                  int32_t D, double p, uint64_t seed, uint64_t offset, const uint64_t *rng,
                  uint32_t flags, const pdssm_strides *strides, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PDSSM_BLOCK_H */
