// C ABI of the MoE layer's training side (moe_train.h): argument checks and the
// launches of each entry point.  Host code only.
#include <float.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "ffn.cuh"
#include "host.cuh"
#include "train.cuh"

namespace {

using moef::aligned;
using moef::cuda_status;
using moef::Gemm;

const uint16_t *u16(const void *p) { return static_cast<const uint16_t *>(p); }
uint16_t *u16(void *p) { return static_cast<uint16_t *>(p); }

bool valid_features(int n) { return n >= 1 && n <= MOEF_MAX_FEATURES; }

// Hidden sizes whose columns the kernels can count past without leaving an int.
constexpr int kMaxHidden = 1 << 30;
bool valid_hidden(int H) { return H >= 1 && H <= kMaxHidden; }

moef_status sms_of_device(int *sms) { return cuda_status(moef::current_sms(sms)); }

// dz and laid out rows of x have a multiple of 8 values, as the dense dz.
int64_t dz_pitch(int64_t cols) { return (cols + 7) / 8 * 8; }

size_t dz_bytes(int64_t P, int64_t cols) { return static_cast<size_t>(P * dz_pitch(cols) * 2); }

// Whether dweight's product can copy x as it lies.
bool lies_in_blocks(const void *x, const int32_t *row_token, int K) {
    return !row_token && K % 8 == 0 && aligned(x, 16);
}

// A product over rows grouped by expert.
moef_status run_group(const Gemm &g, int sms, cudaStream_t stream) {
    cudaError_t err = cudaSuccess;
    const moef::BiasSum none = {};
    if (moef::launch_gemm_tc(g, none, sms, stream, &err)) return cuda_status(err);
    return cuda_status(moef::launch_gemm_simple(g, stream));
}

moef_status expert_backward(const void *dout, const void *x, int64_t T, const int32_t *row_token,
                            const int32_t *offsets, const int32_t *counts, const void *weight,
                            moef_activation act, const void *preact, int gated, void *dx,
                            void *dweight, void *dbias, int64_t P, int E, int n, int K,
                            void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (T < 0 || T > INT_MAX || P < 0 || P > INT_MAX || E < 1 || E > MOEF_MAX_EXPERTS ||
        !valid_features(n) || !valid_features(K))
        return MOEF_ERR_SHAPE;
    if (act < MOEF_ACT_NONE || act > MOEF_ACT_RELU) return MOEF_ERR_ARG;
    if (!row_token && T != P) return MOEF_ERR_SHAPE;
    if (P > 0 && !dx && !dweight && !dbias) return MOEF_ERR_NULL;     // P = 0: dx of no rows
    const bool needs_preact = gated || act != MOEF_ACT_NONE;
    if (!needs_preact && preact) return MOEF_ERR_ARG;
    const int cols = gated ? 2 * n : n;
    const bool copies_x = dweight && !lies_in_blocks(x, row_token, K);
    // dout itself when it is dz and can be copied as it lies
    const bool makes_dz = (dx || dweight) && (needs_preact || cols % 8 || !aligned(dout, 16));
    // without a token or a row there is nothing to read: zeros
    const bool empty = T == 0 || P == 0;
    if (!empty) {
        if (!dout || !offsets || !counts || (needs_preact && !preact) || (dx && !weight) ||
            (dweight && !x) || (!workspace && (makes_dz || copies_x)))
            return MOEF_ERR_NULL;
        if (workspace_bytes <
            moe_expert_backward_workspace_bytes(P, makes_dz ? cols : 0, copies_x ? K : 0))
            return MOEF_ERR_SHAPE;
        if (!aligned(workspace, 16)) return MOEF_ERR_ALIGN;
    }
    for (const void *p : {dout, x, weight, preact, static_cast<const void *>(dx),
                          static_cast<const void *>(dweight), static_cast<const void *>(dbias)})
        if (!aligned(p, 2)) return MOEF_ERR_ALIGN;
    if (!aligned(row_token, 4) || !aligned(offsets, 4) || !aligned(counts, 4))
        return MOEF_ERR_ALIGN;
    moef_status st = MOEF_OK;
    if (empty) {
        const size_t values = static_cast<size_t>(E) * cols * 2;
        if (dweight) st = cuda_status(cudaMemsetAsync(dweight, 0, values * K, stream));
        if (st == MOEF_OK && dbias) st = cuda_status(cudaMemsetAsync(dbias, 0, values, stream));
        return st;
    }
    int sms = 0;
    st = sms_of_device(&sms);
    if (st != MOEF_OK) return st;
    const moef::Groups groups = {offsets, counts, E, P};
    uint16_t *dz = makes_dz ? u16(workspace) : nullptr;
    moef::RowCopy copy = {};
    if (copies_x)
        copy = {u16(x), row_token, u16(workspace) + (dz ? P * dz_pitch(cols) : 0), T, dz_pitch(K),
                K};
    st = cuda_status(moef::launch_expert_dz(u16(dout), u16(preact), static_cast<int>(act), gated,
                                            dz, dz_pitch(cols), u16(dbias), groups, n, copy, sms,
                                            stream));
    Gemm g{};
    g.b = dz ? dz : u16(dout);
    g.b_pitch = dz ? dz_pitch(cols) : cols;
    g.b_rows = P;
    g.a_mn = 1;
    g.M = K;
    g.E = E;
    g.offsets = offsets;
    g.counts = counts;
    if (st == MOEF_OK && dx) {
        Gemm d = g;
        d.a = u16(weight);
        d.N = static_cast<int>(P);
        d.K = cols;
        d.out = dx;
        st = run_group(d, sms, stream);
    }
    if (st == MOEF_OK && dweight) {
        Gemm d = g;
        d.a = copies_x ? copy.to : u16(x);
        d.a_pitch = copies_x ? copy.pitch : K;
        d.a_zeros = copies_x;
        d.b_mn = 1;
        d.b_zeros = dz != nullptr;
        d.N = cols;
        d.K = static_cast<int>(P);
        d.out = dweight;
        st = cuda_status(moef::launch_group_dweight(d, sms, stream));
    }
    return st;
}

// A number of the step, which is taken in fp32.
bool not_negative(double v) { return v >= 0.0 && v <= FLT_MAX; }

}  // namespace

extern "C" {

size_t moe_finalize_backward_workspace_bytes(int T, int H) {
    if (T <= 0 || !valid_hidden(H)) return 0;
    return static_cast<size_t>(moef::finalize_backward_partials(T, H)) * H * sizeof(float);
}

moef_status moe_finalize_backward(const void *permuted_out, int64_t P, const int32_t *idx_map,
                                  const void *weights, moef_weight_kind wkind,
                                  float routed_scale, const void *residual_out,
                                  const void *gamma, float eps, const void *dout,
                                  const void *dresidual_out, const void *dnorm_out,
                                  void *drows, float *dweights, void *dshared, void *dresidual,
                                  void *dgamma, int T, int K, int H, void *workspace,
                                  size_t workspace_bytes, cudaStream_t stream) {
    if (T < 0 || K < 1 || K > MOEF_MAX_K || !valid_hidden(H)) return MOEF_ERR_SHAPE;
    if (wkind != MOEF_W_FP32 && wkind != MOEF_W_BF16 && wkind != MOEF_W_PACKED_TOPK)
        return MOEF_ERR_ARG;
    if (T > 0) {
        if (!drows && !dweights && !dshared && !dresidual && !dgamma) return MOEF_ERR_NULL;
        if (P < 1) return MOEF_ERR_SHAPE;
        if (!idx_map || (drows && !weights) || (dweights && !permuted_out)) return MOEF_ERR_NULL;
        if (!dout && !dresidual_out && !dnorm_out) return MOEF_ERR_NULL;
        if ((dnorm_out != nullptr) != (residual_out != nullptr) ||
            (dnorm_out != nullptr) != (gamma != nullptr) || (dgamma && !dnorm_out))
            return MOEF_ERR_ARG;
        if (dnorm_out && (!(eps >= 0.f) || isinf(eps))) return MOEF_ERR_ARG;
        const size_t need = moe_finalize_backward_workspace_bytes(T, H);
        if (dgamma && need) {
            if (!workspace) return MOEF_ERR_NULL;
            if (workspace_bytes < need) return MOEF_ERR_SHAPE;
            if (!aligned(workspace, 16)) return MOEF_ERR_ALIGN;
        }
    }
    const void *bf16[] = {permuted_out, residual_out, gamma, dout, dresidual_out, dnorm_out,
                          drows, dshared, dresidual, dgamma};
    bool vec = H % 8 == 0;
    for (int i = 0; i < 10; ++i) {
        if (!aligned(bf16[i], 2)) return MOEF_ERR_ALIGN;
        vec = vec && (i == 9 || aligned(bf16[i], 16));
    }
    if (!aligned(idx_map, 4) || !aligned(dweights, 4) ||
        !aligned(weights, wkind == MOEF_W_BF16 ? 2 : 4))
        return MOEF_ERR_ALIGN;
    if (dnorm_out && !moef::finalize_backward_fits(vec ? H / 8 : H)) return MOEF_ERR_SHAPE;
    if (T == 0)
        return dgamma ? cuda_status(cudaMemsetAsync(dgamma, 0, static_cast<size_t>(H) * 2, stream))
                      : MOEF_OK;
    int sms = 0;
    const moef_status st = sms_of_device(&sms);
    if (st != MOEF_OK) return st;
    moef::FinalizeBackward p{};
    p.rows = u16(permuted_out);
    p.P = P;
    p.idx = idx_map;
    p.weights = weights;
    p.wkind = static_cast<int>(wkind);
    p.routed_scale = routed_scale;
    p.r = u16(residual_out);
    p.gamma = u16(gamma);
    p.eps = eps;
    p.dout = u16(dout);
    p.dres = u16(dresidual_out);
    p.dnorm = u16(dnorm_out);
    p.drows = u16(drows);
    p.dweights = dweights;
    p.dshared = u16(dshared);
    p.dresidual = u16(dresidual);
    p.dgamma = u16(dgamma);
    if (dgamma && moef::finalize_backward_partials(T, H))
        p.partial = static_cast<float *>(workspace);
    p.T = T;
    p.K = K;
    p.H = H;
    return cuda_status(moef::launch_finalize_backward(p, sms, stream));
}

moef_status moe_unpermute(const void *rows, int64_t P, const int32_t *idx_map, const void *add0,
                          const void *add1, void *out, int T, int K, int H,
                          cudaStream_t stream) {
    if (T < 0 || P < 0 || K < 1 || K > MOEF_MAX_K || !valid_hidden(H)) return MOEF_ERR_SHAPE;
    if (moef::unpermute_ctas(T, H) > INT_MAX) return MOEF_ERR_SHAPE;
    if (T == 0) return MOEF_OK;
    if ((P > 0 && !rows) || !idx_map || !out) return MOEF_ERR_NULL;
    if (!aligned(rows, 2) || !aligned(add0, 2) || !aligned(add1, 2) || !aligned(out, 2) ||
        !aligned(idx_map, 4))
        return MOEF_ERR_ALIGN;
    moef::Unpermute p{};
    p.rows = u16(rows);
    p.P = P;
    p.idx = idx_map;
    p.add[0] = u16(add0);
    p.add[1] = u16(add1);
    p.out = u16(out);
    p.T = T;
    p.K = K;
    p.H = H;
    return cuda_status(moef::launch_unpermute(p, stream));
}

moef_status moe_topk_route_backward(const float *dweights, const float *weights,
                                    const int32_t *expert_ids, const float *logits, int T,
                                    int E, int K, moef_gate_kind kind, void *dlogits,
                                    moef_out_type out_type, cudaStream_t stream) {
    if (T < 0 || E < 1 || E > MOEF_MAX_EXPERTS || K < 1 || K > MOEF_MAX_K || K > E)
        return MOEF_ERR_SHAPE;
    if ((kind != MOEF_GATE_SOFTMAX && kind != MOEF_GATE_SIGMOID) ||
        (out_type != MOEF_OUT_BF16 && out_type != MOEF_OUT_FP32))
        return MOEF_ERR_ARG;
    if (T == 0) return MOEF_OK;
    if (!dweights || !weights || !expert_ids || !dlogits ||
        (kind == MOEF_GATE_SIGMOID && !logits))
        return MOEF_ERR_NULL;
    if (!aligned(dweights, 4) || !aligned(weights, 4) || !aligned(expert_ids, 4) ||
        !aligned(logits, 4) || !aligned(dlogits, out_type == MOEF_OUT_FP32 ? 4 : 2))
        return MOEF_ERR_ALIGN;
    int sms = 0;
    const moef_status st = sms_of_device(&sms);
    if (st != MOEF_OK) return st;
    const moef::GateBackward p = {dweights, weights, expert_ids, logits, dlogits, T, E, K,
                                  static_cast<int>(kind), out_type == MOEF_OUT_FP32};
    return cuda_status(moef::launch_gate_backward(p, sms, stream));
}

size_t moe_expert_backward_workspace_bytes(int64_t P, int cols, int inputs) {
    if (P < 0 || P > INT_MAX || cols < 0 || cols > 2 * MOEF_MAX_FEATURES || inputs < 0 ||
        inputs > MOEF_MAX_FEATURES)
        return 0;
    return dz_bytes(P, cols) + dz_bytes(P, inputs);
}

moef_status moe_expert_gated_ffn_backward(const void *dout, const void *x, int64_t T,
                                          const int32_t *row_token, const int32_t *offsets,
                                          const int32_t *counts, const void *weight,
                                          moef_activation act, const void *preact, void *dx,
                                          void *dweight, void *dbias, int64_t P, int E, int I,
                                          int H, void *workspace, size_t workspace_bytes,
                                          cudaStream_t stream) {
    return expert_backward(dout, x, T, row_token, offsets, counts, weight, act, preact, 1, dx,
                           dweight, dbias, P, E, I, H, workspace, workspace_bytes, stream);
}

moef_status moe_expert_linear_backward(const void *dout, const void *x, int64_t T,
                                       const int32_t *row_token, const int32_t *offsets,
                                       const int32_t *counts, const void *weight,
                                       moef_activation act, const void *preact, void *dx,
                                       void *dweight, void *dbias, int64_t P, int E, int N,
                                       int K, void *workspace, size_t workspace_bytes,
                                       cudaStream_t stream) {
    return expert_backward(dout, x, T, row_token, offsets, counts, weight, act, preact, 0, dx,
                           dweight, dbias, P, E, N, K, workspace, workspace_bytes, stream);
}

moef_status moe_adamw_step(const moef_adamw_tensor *tensors, int n,
                           const moef_adamw_config *config, cudaStream_t stream) {
    if (!config) return MOEF_ERR_NULL;
    const moef_adamw_config &c = *config;
    if (n < 0) return MOEF_ERR_SHAPE;
    auto beta = [](double b) { return b >= 0.0 && b < 1.0; };
    if (!not_negative(c.lr) || !not_negative(c.eps) || !not_negative(c.weight_decay) || !beta(c.beta1) ||
        !beta(c.beta2) || (!c.device_step && c.step < 1) ||
        (c.state_bits != 8 && c.state_bits != 32) ||
        (c.param_type != MOEF_OUT_BF16 && c.param_type != MOEF_OUT_FP32) ||
        (c.grad_type != MOEF_OUT_BF16 && c.grad_type != MOEF_OUT_FP32))
        return MOEF_ERR_ARG;
    if (n > 0 && !tensors) return MOEF_ERR_NULL;
    if (!aligned(c.device_step, 4) || !aligned(c.device_lr, 4) || !aligned(c.grad_scale, 4))
        return MOEF_ERR_ALIGN;
    const bool eight = c.state_bits == 8;
    int64_t pieces = 0;
    int masters = -1;                   // of the tensors seen so far
    for (int i = 0; i < n; ++i) {
        const moef_adamw_tensor &t = tensors[i];
        if (t.n < 0 || t.n > (int64_t)1 << 40) return MOEF_ERR_SHAPE;
        pieces += (t.n + 255) / 256;
        if (pieces > (int64_t)1 << 31) return MOEF_ERR_SHAPE;
        if (t.n == 0) continue;         // its pointers mean nothing
        if (masters >= 0 && (t.master != nullptr) != masters) return MOEF_ERR_ARG;
        masters = t.master != nullptr;
        if (t.master && c.param_type != MOEF_OUT_BF16) return MOEF_ERR_ARG;
        if (!eight && (t.exp_avg_scale || t.exp_avg_sq_scale)) return MOEF_ERR_ARG;
        if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq ||
            (eight && (!t.exp_avg_scale || !t.exp_avg_sq_scale)))
            return MOEF_ERR_NULL;
        if (!aligned(t.param, c.param_type == MOEF_OUT_FP32 ? 4 : 2) ||
            !aligned(t.grad, c.grad_type == MOEF_OUT_FP32 ? 4 : 2) || !aligned(t.master, 4) ||
            !aligned(t.exp_avg, eight ? 1 : 4) || !aligned(t.exp_avg_sq, eight ? 1 : 4) ||
            !aligned(t.exp_avg_scale, 4) || !aligned(t.exp_avg_sq_scale, 4))
            return MOEF_ERR_ALIGN;
    }
    if (pieces == 0) return MOEF_OK;
    moef::AdamWFactors f{};
    f.beta1 = static_cast<float>(c.beta1);
    f.beta2 = static_cast<float>(c.beta2);
    f.rest1 = static_cast<float>(1.0 - c.beta1);
    f.rest2 = static_cast<float>(1.0 - c.beta2);
    f.eps = static_cast<float>(c.eps);
    f.lr = static_cast<float>(c.lr);
    f.weight_decay = static_cast<float>(c.weight_decay);
    // log(0) = -inf gives 1 - beta^step = 1
    const double log1 = log(c.beta1), log2 = log(c.beta2);
    const int step = c.device_step ? 1 : c.step;
    f.log_beta1 = static_cast<float>(log1);
    f.log_beta2 = static_cast<float>(log2);
    f.bias1 = static_cast<float>(-expm1(step * log1));
    f.root_bias2 = static_cast<float>(sqrt(-expm1(step * log2)));
    f.device_step = c.device_step;
    f.device_lr = c.device_lr;
    f.grad_scale = c.grad_scale;
    return cuda_status(moef::launch_adamw(tensors, n, f, c.state_bits, masters,
                                          c.param_type == MOEF_OUT_FP32,
                                          c.grad_type == MOEF_OUT_FP32, stream));
}

}  // extern "C"
