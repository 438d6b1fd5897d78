/*
 * moe_train.h -- C ABI of the MoE layer's training side (libmoe_finalize.so),
 * hand-written CUDA for sm_103a: the gradients of the deferred finalize, of the
 * row gather in front of the experts, of the top-K gate and of the expert
 * products, and an AdamW step over many tensors.  With moe_linear_backward
 * and moe_gated_ffn_backward (moe_ffn.h) the whole layer can be trained:
 *
 *   drows, dweights, dshared  = moe_finalize_backward(dout)
 *   dh, dw2                   = moe_expert_linear_backward(drows)
 *   dxr, dw13                 = moe_expert_gated_ffn_backward(dh)
 *   dlogits                   = moe_topk_route_backward(dweights)
 *   dx                        = moe_unpermute(dxr) + the router's and the shared expert's
 *   weights                   = moe_adamw_step(gradients)
 *
 * Conventions are those of moe_finalize.h and moe_ffn.h: device pointers, bf16
 * as raw bit patterns, dense row-major arrays, the caller owns every buffer,
 * nothing is allocated or synchronised, work is enqueued on `stream` of the
 * current device, argument errors are returned before anything is enqueued,
 * and a call may be captured in a CUDA graph (make one of each kind before a
 * capture).  Kernels are programmatic dependents of the previous kernel on
 * the stream.  Sums run in fp32 in a fixed order: equal calls give equal bits.
 * Workspaces hold nothing between calls; calls that may run at the same time
 * need one each.
 *
 * Outputs must not overlap inputs or each other, except where an entry point
 * says so.
 */
#ifndef MOE_TRAIN_H_
#define MOE_TRAIN_H_

#include "moe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_finalize_backward -- gradients of moe_finalize.  With inv[t] =
 * (mean_h residual_out[t,h]^2 + eps)^(-1/2) and r = residual_out:
 *
 *   dr[t,h]   = dresidual_out[t,h] + inv (dnorm_out[t,h] gamma[h]
 *               - r[t,h] inv^2 mean_h(dnorm_out gamma r))
 *   dm[t,h]   = dout[t,h] + dr[t,h]
 *   drows[idx[t,k], h] = w[t,k] routed_scale dm[t,h]
 *   dweights[t,k]      = routed_scale sum_h dm[t,h] permuted_out[idx[t,k], h]
 *   dshared = dm,  dresidual = dr,  dgamma[h] = sum_t dnorm_out[t,h] r[t,h] inv[t]
 *
 * (the rounding of residual_out counts as the identity).
 *
 *   permuted_out, P, idx_map, weights, wkind, routed_scale, gamma, eps, T, K, H
 *                  as in the forward call; weights may be NULL without drows,
 *                  permuted_out without dweights
 *   residual_out   bf16 [T, H] as the forward call wrote it; required with
 *                  dnorm_out, as gamma is, and else NULL, as gamma is
 *   dout, dresidual_out, dnorm_out
 *                  bf16 [T, H], the outputs' gradients; NULL is zero (at
 *                  least one non-NULL)
 *   drows          bf16 [P, H] or NULL; rows that no slot names are left as
 *                  they were
 *   dweights       fp32 [T, K] or NULL
 *   dshared, dresidual  bf16 [T, H], each or NULL (equal values without dout)
 *   dgamma         bf16 [H] or NULL; needs dnorm_out
 *                  (at least one output non-NULL when T > 0)
 *   workspace      moe_finalize_backward_workspace_bytes(T, H) bytes with
 *                  dgamma, 16-byte aligned, contents irrelevant; may be NULL
 *                  without dgamma or when that is 0 (up to 32 tokens, 16
 *                  if H % 8 != 0)
 *
 * A slot whose idx_map is outside [0, P) has no row: its dweights is 0.  No two
 * slots may name the same row.  dm stays in fp32 up to each output's rounding.
 * In place: dshared or dresidual may equal dout or dresidual_out.
 * T = 0 writes zeros to dgamma.  1 <= H <= 2^30.  MOEF_ERR_SHAPE when a row is
 * too long for one cluster: with dnorm_out, more than 32768 pieces of 8 values (of single
 * values, where H % 8 != 0 or a pointer is not 16-byte aligned).
 */
size_t moe_finalize_backward_workspace_bytes(int T, int H);

moef_status moe_finalize_backward(const void *permuted_out, int64_t P, const int32_t *idx_map,
                                  const void *weights, moef_weight_kind wkind,
                                  float routed_scale, const void *residual_out,
                                  const void *gamma, float eps, const void *dout,
                                  const void *dresidual_out, const void *dnorm_out,
                                  void *drows, float *dweights, void *dshared, void *dresidual,
                                  void *dgamma, int T, int K, int H, void *workspace,
                                  size_t workspace_bytes, cudaStream_t stream);

/*
 * moe_unpermute -- rows grouped by expert back to their tokens, summed:
 *
 *   out[t,h] = sum_k rows[idx_map[t,k], h] + add0[t,h] + add1[t,h]
 *
 * the gradient of the row gather in front of the experts (a token's row goes
 * to each of its experts) plus what reaches the token on other ways.
 *
 *   rows     bf16 [P, H];  idx_map int32 [T, K] as from moe_permute: a slot
 *            outside [0, P) adds nothing
 *   add0, add1   bf16 [T, H], each or NULL;  out bf16 [T, H], may equal either
 *            (MOEF_ERR_SHAPE when T ceil(H / 128) passes INT_MAX)
 *   P >= 0 (rows may be NULL with P = 0), T >= 0 (0 enqueues nothing),
 *   1 <= K <= MOEF_MAX_K, 1 <= H <= 2^30
 */
moef_status moe_unpermute(const void *rows, int64_t P, const int32_t *idx_map, const void *add0,
                          const void *add1, void *out, int T, int K, int H,
                          cudaStream_t stream);

/*
 * moe_topk_route_backward -- gradients of moe_topk_route's weights, into the
 * logits of the chosen experts (the choice itself has none):
 *
 *   d[t,k]  = weights[t,k] (dweights[t,k] - sum_j weights[t,j] dweights[t,j])
 *   SOFTMAX: dlogits[t, ids[t,k]] = d[t,k]
 *   SIGMOID: dlogits[t, ids[t,k]] = d[t,k] (1 - s(logits[t, ids[t,k]]))
 *   dlogits = 0 elsewhere
 *
 *   dweights, weights  fp32 [T, K];  expert_ids int32 [T, K]; a slot whose id
 *                      is outside [0, E) counts in no sum
 *   logits   fp32 [T, E] as in the forward call; NULL for MOEF_GATE_SOFTMAX
 *   dlogits  [T, E], bf16 or fp32 by out_type
 *   sizes as in moe_topk_route.  A token that names an expert twice gets the sum.
 */
moef_status moe_topk_route_backward(const float *dweights, const float *weights,
                                    const int32_t *expert_ids, const float *logits, int T,
                                    int E, int K, moef_gate_kind kind, void *dlogits,
                                    moef_out_type out_type, cudaStream_t stream);

/*
 * moe_expert_gated_ffn_save / moe_expert_linear_save -- moe_expert_gated_ffn
 * and moe_expert_linear that also keep the preactivations for the backward
 * pass: preact bf16 [P, 2I] ([P, N]), rows of no expert left as they were.
 */
moef_status moe_expert_gated_ffn_save(const void *x, int64_t T, const int32_t *row_token,
                                      const int32_t *offsets, const int32_t *counts,
                                      const void *weight, const void *bias,
                                      moef_activation act, void *out, void *preact, int64_t P,
                                      int E, int I, int H, cudaStream_t stream);

moef_status moe_expert_linear_save(const void *x, int64_t T, const int32_t *row_token,
                                   const int32_t *offsets, const int32_t *counts,
                                   const void *weight, const void *bias, moef_activation act,
                                   void *out, void *preact, int64_t P, int E, int N, int K,
                                   cudaStream_t stream);

/*
 * moe_expert_gated_ffn_backward / moe_expert_linear_backward -- gradients of
 * the expert products for dout = dL/d out.  With dz as in
 * moe_gated_ffn_backward (moe_linear_backward) and R_e the rows of expert e:
 *
 *   dx[r,:]        = dz[r,:] weight[e]                         r in R_e
 *   dweight[e]     = sum over r in R_e of dz[r,:]^T x[row_token[r],:]
 *   dbias[e]       = sum over r in R_e of dz[r,:]
 *
 *   dout, preact   bf16 [P, I], [P, 2I] ([P, N] each; preact required unless
 *                  act is MOEF_ACT_NONE, then NULL)
 *   x, T, row_token, offsets, counts, weight, E   as in the forward call; x
 *                  may be NULL without dweight, weight without dx
 *   dx             bf16 [P, H] ([P, K]) or NULL: per row, also with row_token
 *                  (moe_unpermute sums them to tokens); rows of no expert are
 *                  left as they were
 *   dweight        bf16 [E, 2I, H] ([E, N, K]) or NULL; zeros for an expert
 *                  without rows
 *   dbias          bf16 [E, 2I] ([E, N]) or NULL          (at least one non-NULL when P > 0)
 *   workspace      moe_expert_backward_workspace_bytes(P, cols, inputs) bytes,
 *                  16-byte aligned (NULL when that is 0): cols the width of dz
 *                  (2I, or N), 0 when dout is dz and lies so that it can be
 *                  copied (linear without an activation, N a multiple of 8, dout
 *                  16-byte aligned) or neither dx nor dweight is wanted; inputs
 *                  the width of x (H, or K) when dweight is wanted and x cannot
 *                  be copied as it lies (with row_token, when the width is not a
 *                  multiple of 8, or x not 16-byte aligned), else 0
 *
 * With T or P 0 dweight and dbias are zeros and nothing else is done.  Rows of
 * no expert are read by nothing that counts: they may hold anything.
 * Rows at or past P, and experts whose offset is negative, take no part.  dz
 * is rounded to bf16 for the two products; dbias sums it before that.  A
 * row_token outside [0, T) counts as a row of zeros in dweight.
 */
size_t moe_expert_backward_workspace_bytes(int64_t P, int cols, int inputs);

moef_status moe_expert_gated_ffn_backward(const void *dout, const void *x, int64_t T,
                                          const int32_t *row_token, const int32_t *offsets,
                                          const int32_t *counts, const void *weight,
                                          moef_activation act, const void *preact, void *dx,
                                          void *dweight, void *dbias, int64_t P, int E, int I,
                                          int H, void *workspace, size_t workspace_bytes,
                                          cudaStream_t stream);

moef_status moe_expert_linear_backward(const void *dout, const void *x, int64_t T,
                                       const int32_t *row_token, const int32_t *offsets,
                                       const int32_t *counts, const void *weight,
                                       moef_activation act, const void *preact, void *dx,
                                       void *dweight, void *dbias, int64_t P, int E, int N,
                                       int K, void *workspace, size_t workspace_bytes,
                                       cudaStream_t stream);

/*
 * moe_adamw_step -- one AdamW step (decoupled weight decay) over a list of
 * tensors, in as few launches as their table allows (one for each 256):
 *
 *   g  = grad_scale grad
 *   m  = beta1 m + (1 - beta1) g
 *   v  = beta2 v + (1 - beta2) g^2
 *   p  = p (1 - lr weight_decay)
 *        - lr / (1 - beta1^step) * m / (sqrt(v / (1 - beta2^step)) + eps)
 *
 * in fp32, in place.  tensors: a HOST array of n descriptions, read during the
 * call only; the element types are the call's:
 *   param   param_type (MOEF_OUT_BF16 or MOEF_OUT_FP32) [n], read and written
 *   master  fp32 [n]: the value that is updated, param then receives its
 *           rounding (and is not read); with bf16 params only; NULL for all
 *           tensors or for none
 *   grad    grad_type [n]
 *   exp_avg, exp_avg_sq   state_bits 32: fp32 m and v [n], the scales NULL.
 *           state_bits 8: e4m3 values [n] and fp32 scales [ceil(n / 256)], one
 *           for each 256 values in order: m = exp_avg scale, and sqrt(v) =
 *           exp_avg_sq scale.  A scale is the largest magnitude of its values
 *           divided by 448; sqrt(v) > 0 is never stored as 0 (its least code is
 *           2^-9 scale), so that no step divides by eps alone where there was a
 *           gradient.  The step itself uses m and v before they are rounded.
 *   n       values, >= 0 (0: its pointers are ignored)
 * No array may overlap another, nor two tensors share one.  Zeros are the
 * states before the first step.
 *
 * step >= 1 counts this step.  Device values, each NULL or one number that the
 * kernels read when they run, so that a captured step can be replayed with
 * others: device_step (int32, in place of step; below 1 it counts as 1),
 * device_lr (in place of lr), grad_scale (NULL: 1; the factor of a clipped norm
 * or of a scaled loss).
 *
 * Alignment: 16 bytes (8 bits: 8 for the states) of all of a tensor's arrays
 * allow 16-byte accesses; others take single values.  A v that passes the largest
 * fp32 number (a scaled gradient above 1.8e19 can) is infinite, and the value moves by
 * its decay alone: for good with fp32 states, while 8 bits store a sqrt(v) of 2^64
 * (1 - 2^-20) at most, which decays again.  A gradient that is not
 * finite leaves its value and its fp32 states not finite.  With 8 bits, NaN is its own
 * value's alone in both states; an infinite one makes all 256 values of exp_avg NaN
 * (their scale is infinite), while its sqrt(v) is stored as the largest above, beside
 * which the block's other roots keep the least code above 0.
 * MOEF_ERR_ARG for lr, eps or weight_decay negative or not finite in fp32, a beta
 * outside [0, 1), step < 1 without device_step, or state_bits other than 8
 * and 32.  tensors may be NULL with n = 0.
 */
typedef struct {
    void *param;
    float *master;
    const void *grad;
    void *exp_avg, *exp_avg_sq;
    float *exp_avg_scale, *exp_avg_sq_scale;
    int64_t n;
} moef_adamw_tensor;

typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    const int32_t *device_step;
    const float *device_lr, *grad_scale;
    int step;
    int state_bits;
    moef_out_type param_type, grad_type;
} moef_adamw_config;

moef_status moe_adamw_step(const moef_adamw_tensor *tensors, int n,
                           const moef_adamw_config *config, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAIN_H_ */
