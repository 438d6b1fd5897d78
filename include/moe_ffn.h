/*
 * moe_ffn.h -- C ABI of the matrix products around the deferred MoE finalize
 * (libmoe_finalize.so), hand-written CUDA for sm_103a.
 *
 * moe_finalize (moe_finalize.h) reads three things that other kernels make:
 * the routing weights and row map of the gate, the unweighted, permuted
 * expert rows, and the shared-expert output.  The entry points here make
 * them from a layer's input x [T, H]:
 *
 *   logits        = moe_linear(x, w_router)            fp32 [T, E]
 *   ids, weights  = moe_topk_route(logits)
 *   row map       = moe_permute(ids)
 *   h             = moe_expert_gated_ffn(x, row map)   bf16 [P, I]
 *   permuted_out  = moe_expert_linear(h)               bf16 [P, H]
 *   hs            = moe_gated_ffn(x)                   bf16 [T, I]
 *   shared_out    = moe_linear(hs, w_down)             bf16 [T, H]
 *   out           = moe_finalize(permuted_out, row map, weights, shared_out)
 *
 * moe_linear and moe_gated_ffn also have their backward passes; those of the
 * expert products, the gate and the finalize are in moe_train.h.
 *
 * Conventions are those of moe_finalize.h: device pointers, bf16 as raw bit
 * patterns, dense row-major arrays, the caller owns every buffer, nothing is
 * allocated or synchronised, work is enqueued on `stream` of the current
 * device, argument errors are returned before anything is enqueued, and a
 * call may be captured in a CUDA graph.  No call keeps state between calls.
 * The first call on a device looks up launch limits and sets kernel
 * attributes; make one of each kind before a capture.  Kernels are launched as
 * programmatic dependents of the previous kernel on the stream, as in
 * moe_finalize.h, and touch no global memory before it has completed.
 *
 * Arithmetic: products of bf16 values are summed in fp32; bias, activation,
 * gate product and residual are applied to the unrounded sum, and each output
 * is rounded once, to nearest even.
 *
 * Alignment: bf16 pointers must be 2-byte aligned, fp32 and int32 pointers
 * 4-byte aligned (else MOEF_ERR_ALIGN).  The tensor-core path is used when
 * every matrix operand is 16-byte aligned with rows of a multiple of 8
 * values; any other case takes a slower path of single-value loads with the
 * same results up to the order of the sums.  (The number of output features
 * may be odd on either path; moe_linear_backward's inputs K decide for it.)
 *
 * Outputs must not overlap inputs, except where an entry point says so.
 */
#ifndef MOE_FFN_H_
#define MOE_FFN_H_

#include "moe_finalize.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations a(z):
 *   NONE       z
 *   SILU       z / (1 + exp(-z))
 *   GELU       z * Phi(z), Phi the standard normal distribution function
 *   GELU_TANH  0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))
 *   RELU       max(z, 0); its derivative at 0 is 0                          */
typedef enum {
    MOEF_ACT_NONE = 0,
    MOEF_ACT_SILU = 1,
    MOEF_ACT_GELU = 2,
    MOEF_ACT_GELU_TANH = 3,
    MOEF_ACT_RELU = 4
} moef_activation;

/* Largest feature count (N, K, I, H) accepted. */
#define MOEF_MAX_FEATURES (1 << 24)

/* Element type of an output. */
typedef enum { MOEF_OUT_BF16 = 0, MOEF_OUT_FP32 = 1 } moef_out_type;

/*
 * moe_linear -- matrix product with bias, activation and residual:
 *
 *   z[t,n]   = sum_k x[t,k] * weight[n,k] + bias[n]
 *   out[t,n] = act(z[t,n]) + residual[t,n]
 *
 *   x         bf16 [T, K]
 *   weight    bf16 [N, K]
 *   bias      bf16 [N], or NULL (0)
 *   residual  bf16 [T, N], or NULL (0)
 *   out       [T, N], bf16 or fp32 by out_type
 *   preact    bf16 [T, N], or NULL: receives bf16(z) for the backward pass
 *   T         rows (>= 0; T = 0 returns MOEF_OK and enqueues nothing)
 *   N, K      1 .. MOEF_MAX_FEATURES
 *
 * In place: a bf16 out may equal residual.
 */
moef_status moe_linear(const void *x, const void *weight, const void *bias,
                       const void *residual, moef_activation act, void *out,
                       moef_out_type out_type, void *preact, int T, int N, int K,
                       cudaStream_t stream);

/*
 * moe_linear_backward -- gradients of moe_linear for dout = dL/d out:
 *
 *   dz[t,n]      = dout[t,n] * act'(preact[t,n])
 *   dx[t,k]      = sum_n dz[t,n] * weight[n,k]
 *   dweight[n,k] = sum_t dz[t,n] * x[t,k]
 *   dbias[n]     = sum_t dz[t,n]
 *   (the gradient of the residual is dout itself)
 *
 *   dout, preact  bf16 [T, N]; preact as moe_linear wrote it, required
 *                 unless act is MOEF_ACT_NONE (then NULL)
 *   x, weight     as in the forward call; x may be NULL without dweight,
 *                 weight without dx
 *   dx            bf16 [T, K] or NULL    dweight  bf16 [N, K] or NULL
 *   dbias         bf16 [N] or NULL       (at least one non-NULL)
 *   workspace     moe_linear_backward_workspace_bytes(T, N) bytes, 16-byte
 *                 aligned, contents irrelevant; calls that may run at the
 *                 same time need one each
 *
 * dz is rounded to bf16 for the two products (they run on the tensor cores);
 * dbias sums it before that rounding.  All sums run in a fixed order: equal
 * calls give equal bits.  T = 0 writes zeros to dweight and dbias.
 */
size_t moe_linear_backward_workspace_bytes(int T, int N);

moef_status moe_linear_backward(const void *dout, const void *x, const void *weight,
                                moef_activation act, const void *preact,
                                void *dx, void *dweight, void *dbias, int T, int N, int K,
                                void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * moe_gated_ffn -- the gated feed-forward block, both projections, the
 * activation and the product in one kernel:
 *
 *   z[t,j]   = sum_k x[t,k] * weight[j,k] + bias[j]          0 <= j < 2I
 *   out[t,i] = act(z[t,i]) * z[t,I+i]                        0 <= i < I
 *
 *   x         bf16 [T, H]
 *   weight    bf16 [2I, H]: I rows of the gate projection, then I of the up
 *             projection
 *   bias      bf16 [2I], or NULL
 *   out       bf16 [T, I]
 *   preact    bf16 [T, 2I], or NULL: receives bf16(z) for the backward pass
 *   T >= 0; I, H 1 .. MOEF_MAX_FEATURES
 */
moef_status moe_gated_ffn(const void *x, const void *weight, const void *bias,
                          moef_activation act, void *out, void *preact,
                          int T, int I, int H, cudaStream_t stream);

/*
 * moe_gated_ffn_backward -- gradients of moe_gated_ffn for dout = dL/d out,
 * with g = preact[:, :I] and u = preact[:, I:]:
 *
 *   dz[t,i]   = dout[t,i] * u[t,i] * act'(g[t,i])
 *   dz[t,I+i] = dout[t,i] * act(g[t,i])
 *   dx = dz weight,   dweight = dz^T x,   dbias = column sums of dz
 *
 *   dout bf16 [T, I]; preact bf16 [T, 2I] as moe_gated_ffn wrote it;
 *   dx bf16 [T, H], dweight bf16 [2I, H], dbias bf16 [2I], each or NULL
 *   workspace: moe_gated_ffn_backward_workspace_bytes(T, I) bytes
 *
 * Otherwise as moe_linear_backward.
 */
size_t moe_gated_ffn_backward_workspace_bytes(int T, int I);

moef_status moe_gated_ffn_backward(const void *dout, const void *x, const void *weight,
                                   moef_activation act, const void *preact,
                                   void *dx, void *dweight, void *dbias, int T, int I, int H,
                                   void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * moe_permute -- the padded, expert-grouped layout of T x K routing slots:
 *
 *   expert_ids  int32 [T, K]; an id outside [0, E) marks a slot without a row
 *               (a padding token of the batch, an expert of another rank)
 *   tile        each expert's rows are padded up to a multiple of tile (>= 1)
 *   idx_map     int32 [T, K]: the slot's row, or -1 for a slot without one.
 *               moe_finalize needs every entry in [0, P): pass it the tokens
 *               whose slots all have rows (padding at the end of a batch: a
 *               smaller T); moe_finalize_check_indices counts the others
 *   row_token   int32 [P]: the token of each row, -1 on padding rows
 *   P           rows of row_token, at least moe_permute_rows(T, K, E, tile)
 *   offsets     int32 [E + 1]: each expert's first row (a multiple of tile);
 *               offsets[E] is the end of the last expert's rows
 *   counts      int32 [E]: each expert's rows without padding
 *   workspace   moe_permute_workspace_bytes(T, K, E) bytes, 16-byte aligned,
 *               contents irrelevant; may be NULL when that is 0 (up to 16384
 *               slots)
 *
 * Experts stand in ascending order, an expert's rows in (token, slot) order;
 * all outputs are exact.  P may exceed that number; all P rows are written.  A
 * token may name an expert twice; it gets two rows.
 * 1 <= K <= MOEF_MAX_K, 1 <= E <= MOEF_MAX_EXPERTS, T >= 0 (T = 0 writes zero
 * offsets and counts and -1 to row_token).
 *
 * moe_permute_rows -- the most rows any routing can need; the host cannot
 * know the actual number without waiting for the device.  0 when a size is
 * out of range or the number does not fit in 31 bits.
 */
int64_t moe_permute_rows(int T, int K, int E, int tile);

size_t moe_permute_workspace_bytes(int T, int K, int E);

moef_status moe_permute(const int32_t *expert_ids, int T, int K, int E, int tile,
                        int32_t *idx_map, int32_t *row_token, int64_t P,
                        int32_t *offsets, int32_t *counts,
                        void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * moe_expert_gated_ffn / moe_expert_linear -- the gated block and the linear
 * product over rows grouped by expert: row r of expert e, offsets[e] <= r <
 * offsets[e] + counts[e], is computed with expert e's weights from row
 * row_token[r] of x (row r of x without row_token).
 *
 *   x          bf16 [T, H] ([T, K])
 *   row_token  int32 [P], or NULL: then x is in the layout itself, T = P
 *   offsets    int32 [E + 1], counts int32 [E], as from moe_permute
 *   weight     bf16 [E, 2I, H] ([E, N, K])
 *   bias       bf16 [E, 2I] ([E, N]), or NULL
 *   out        bf16 [P, I] ([P, N]); rows of no expert are left as they were
 *   T, P       0 .. INT_MAX; with either 0 nothing is enqueued
 *   E          1 .. MOEF_MAX_EXPERTS
 *
 * The layout is read on the device.  Rows at or past P are not computed, and
 * a row_token outside [0, T) reads as a row of zeros.
 */
moef_status moe_expert_gated_ffn(const void *x, int64_t T, const int32_t *row_token,
                                 const int32_t *offsets, const int32_t *counts,
                                 const void *weight, const void *bias, moef_activation act,
                                 void *out, int64_t P, int E, int I, int H,
                                 cudaStream_t stream);

moef_status moe_expert_linear(const void *x, int64_t T, const int32_t *row_token,
                              const int32_t *offsets, const int32_t *counts,
                              const void *weight, const void *bias, moef_activation act,
                              void *out, int64_t P, int E, int N, int K,
                              cudaStream_t stream);

/*
 * moe_ffn_lost_waits -- health check of the tensor-core kernels.  Their warps
 * hand work to each other through barriers; a wait that has not ended after
 * two seconds, and 2 us more for each 64 values of k summed meanwhile (which no
 * correct run comes near: 0.5 us at most), is given up, the launch ends with
 * undefined outputs, and the count kept here for the current device goes up.
 * Writes the count since the library was loaded; waits for the device (call it
 * outside the hot path, not during a capture).
 */
moef_status moe_ffn_lost_waits(unsigned *count);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FFN_H_ */
