// Declarations shared by the translation units of the MoE layer's training
// side (moe_train.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_train.h"

namespace moef {

// Gradients of the finalize; null pointers as in moe_finalize_backward.
struct FinalizeBackward {
    const uint16_t *rows;               // bf16 [P, H]
    int64_t P;
    const int32_t *idx;                 // [T, K]
    const void *weights;                // [T, K], encoding in wkind
    int wkind;
    float routed_scale;
    const uint16_t *r, *gamma;          // residual_out [T, H], [H]
    float eps;
    const uint16_t *dout, *dres, *dnorm;
    uint16_t *drows;
    float *dweights;
    uint16_t *dshared, *dresidual, *dgamma;
    float *partial;                     // fp32 [clusters, H] when dgamma needs it
    int T, K, H;
};

// Rows of partial that a launch can need; and whether a row fits.
int finalize_backward_partials(int T, int H);
bool finalize_backward_fits(int64_t nvec);
cudaError_t launch_finalize_backward(const FinalizeBackward &p, int num_sms, cudaStream_t stream);

struct Unpermute {
    const uint16_t *rows;
    int64_t P;
    const int32_t *idx;
    const uint16_t *add[2];             // each may be null
    uint16_t *out;
    int T, K, H;
};
int64_t unpermute_ctas(int T, int H);       // at most: a launch takes INT_MAX
cudaError_t launch_unpermute(const Unpermute &p, cudaStream_t stream);

struct GateBackward {
    const float *dweights, *weights;
    const int32_t *ids;
    const float *logits;
    void *dlogits;
    int T, E, K, kind, f32;
};
cudaError_t launch_gate_backward(const GateBackward &p, int num_sms, cudaStream_t stream);

// What a step multiplies with; the device pointers as in moef_adamw_config.
struct AdamWFactors {
    float beta1, beta2, rest1, rest2;   // rest: 1 - beta
    float eps, lr, weight_decay;
    float bias1, root_bias2;            // 1 - beta1^step, sqrt(1 - beta2^step)
    float log_beta1, log_beta2;         // for device_step
    const int32_t *device_step;
    const float *device_lr, *grad_scale;
};
cudaError_t launch_adamw(const moef_adamw_tensor *tensors, int n, const AdamWFactors &f,
                         int state_bits, int masters, int param_f32, int grad_f32,
                         cudaStream_t stream);

// dz of the expert products over the rows of the experts alone, the rows of x that
// they were made from laid out beside it, and dbias.
struct Groups {
    const int32_t *offsets, *counts;
    int E;
    int64_t P;
};
struct RowCopy {
    const uint16_t *x;          // [T, K]
    const int32_t *row_token;   // [P], or null: row r of x
    uint16_t *to;               // [P, pitch], null: nothing to do
    int64_t T, pitch;
    int K;
};
cudaError_t launch_expert_dz(const uint16_t *dout, const uint16_t *preact, int act, int gated,
                             uint16_t *dz, int64_t pitch, uint16_t *dbias,
                             const Groups &groups, int n, const RowCopy &copy, int num_sms,
                             cudaStream_t stream);

}  // namespace moef
