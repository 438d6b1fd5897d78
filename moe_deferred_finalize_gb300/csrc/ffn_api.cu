// C ABI of the matrix products around the finalize (moe_ffn.h): argument
// checks and the launches of each entry point.  Host code only.
#include <limits.h>
#include <stdint.h>

#include "ffn.cuh"
#include "host.cuh"
#include "internal.cuh"

namespace {

using moef::aligned;
using moef::cuda_status;
using moef::Gemm;

bool valid_act(moef_activation a) { return a >= MOEF_ACT_NONE && a <= MOEF_ACT_RELU; }

bool valid_features(int n) { return n >= 1 && n <= MOEF_MAX_FEATURES; }

const uint16_t *u16(const void *p) { return static_cast<const uint16_t *>(p); }

// dz has rows of a multiple of 8 values, so that the tensor-core kernels can
// copy it whatever the number of features is.
int64_t dz_pitch(int64_t cols) { return (cols + 7) / 8 * 8; }

size_t dz_bytes(int64_t T, int64_t cols) { return static_cast<size_t>(T * dz_pitch(cols) * 2); }

size_t backward_bytes(int64_t T, int64_t cols) {
    const int64_t rows = T > 0 ? (T - 1) / moef::sum_rows(static_cast<int>(T)) + 1 : 0;
    return dz_bytes(T, cols) + static_cast<size_t>(rows * cols * 4);
}

// One product, and the bias gradient that goes with it (taken out of *bias).
moef_status run_gemm(const Gemm &g, moef::BiasSum *bias, cudaStream_t stream) {
    int sms = 0;
    const moef_status st = cuda_status(moef::current_sms(&sms));
    if (st != MOEF_OK) return st;
    cudaError_t err = cudaSuccess;
    if (moef::launch_gemm_decode(g, sms, stream, &err)) return cuda_status(err);
    if (moef::launch_gemm_tc(g, *bias, sms, stream, &err)) {
        bias->dbias = nullptr;
        return cuda_status(err);
    }
    return cuda_status(moef::launch_gemm_simple(g, stream));
}

// The backward pass of z = x weight^T + bias with `cols` features z, from
// dout [T, n] (n = cols, or cols / 2 when gated) and preact [T, cols].
moef_status backward(const void *dout, const void *x, const void *weight, moef_activation act,
                     const void *preact, int gated, void *dx, void *dweight, void *dbias, int T,
                     int n, int K, void *workspace, size_t workspace_bytes,
                     cudaStream_t stream) {
    if (T < 0 || !valid_features(n) || !valid_features(K)) return MOEF_ERR_SHAPE;
    const int cols = gated ? 2 * n : n;
    if (!valid_act(act)) return MOEF_ERR_ARG;
    if (!dx && !dweight && !dbias) return MOEF_ERR_NULL;
    const bool needs_preact = gated || act != MOEF_ACT_NONE;
    if (!needs_preact && preact) return MOEF_ERR_ARG;
    if (T > 0) {
        if (!dout || (needs_preact && !preact) || (dx && !weight) || (dweight && !x))
            return MOEF_ERR_NULL;
        if (!workspace) return MOEF_ERR_NULL;
        if (workspace_bytes < backward_bytes(T, cols)) return MOEF_ERR_SHAPE;
        if (!aligned(workspace, 16)) return MOEF_ERR_ALIGN;
    }
    if (!aligned(dout, 2) || !aligned(x, 2) || !aligned(weight, 2) || !aligned(preact, 2) ||
        !aligned(dx, 2) || !aligned(dweight, 2) || !aligned(dbias, 2))
        return MOEF_ERR_ALIGN;
    if (T == 0) {
        moef_status st = MOEF_OK;
        if (dweight)
            st = cuda_status(cudaMemsetAsync(dweight, 0, static_cast<size_t>(cols) * K * 2,
                                             stream));
        if (st == MOEF_OK && dbias)
            st = cuda_status(cudaMemsetAsync(dbias, 0, static_cast<size_t>(cols) * 2, stream));
        return st;
    }
    // dout itself when it is dz and can be copied as it lies
    const bool has_dz = needs_preact || cols % 8 || !aligned(dout, 16);
    uint16_t *dz = has_dz && (dx || dweight) ? static_cast<uint16_t *>(workspace) : nullptr;
    float *partial = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                               dz_bytes(T, cols));
    if (dz || dbias) {
        const moef_status st = cuda_status(moef::launch_dz(
            u16(dout), u16(preact), static_cast<int>(act), gated, dz, dz_pitch(cols),
            dbias ? partial : nullptr, T, n, stream));
        if (st != MOEF_OK) return st;
    }
    moef::BiasSum bias = {partial, static_cast<uint16_t *>(dbias),
                          (T - 1) / moef::sum_rows(T) + 1, cols};
    Gemm g[2] = {};
    int n_products = 0;
    if (dx) {
        Gemm &x_grad = g[n_products++];
        x_grad.a = u16(weight);
        x_grad.a_mn = 1;
        x_grad.M = K;
        x_grad.N = T;
        x_grad.K = cols;
        x_grad.out = dx;
        x_grad.b_rows = T;
    }
    if (dweight) {
        Gemm &w_grad = g[n_products++];
        w_grad.a = u16(x);
        w_grad.a_mn = 1;
        w_grad.b_mn = 1;
        w_grad.M = K;
        w_grad.N = cols;
        w_grad.K = T;
        w_grad.out = dweight;
        w_grad.b_rows = cols;
    }
    for (int i = 0; i < n_products; ++i) {
        g[i].b = dz ? dz : u16(dout);
        g[i].b_pitch = dz ? dz_pitch(cols) : cols;
    }
    if (n_products == 2) {
        int sms = 0;
        const moef_status st = cuda_status(moef::current_sms(&sms));
        if (st != MOEF_OK) return st;
        cudaError_t err = cudaSuccess;
        if (moef::launch_two_gemms_tc(g, bias, sms, stream, &err)) return cuda_status(err);
    }
    for (int i = 0; i < n_products; ++i) {
        const moef_status st = run_gemm(g[i], &bias, stream);
        if (st != MOEF_OK) return st;
    }
    return cuda_status(moef::launch_bias_sum(bias, stream));
}

moef_status expert_product(const void *x, int64_t T, const int32_t *row_token,
                           const int32_t *offsets, const int32_t *counts, const void *weight,
                           const void *bias, moef_activation act, int gated, void *out,
                           int64_t P, int E, int M, int K, cudaStream_t stream) {
    if (T < 0 || T > INT_MAX || P < 0 || P > INT_MAX || E < 1 || E > MOEF_MAX_EXPERTS ||
        !valid_features(M) || !valid_features(K))
        return MOEF_ERR_SHAPE;
    if (!valid_act(act)) return MOEF_ERR_ARG;
    if (!row_token && T != P) return MOEF_ERR_SHAPE;
    if (T == 0 || P == 0) return MOEF_OK;
    if (!x || !offsets || !counts || !weight || !out) return MOEF_ERR_NULL;
    if (!aligned(x, 2) || !aligned(weight, 2) || !aligned(bias, 2) || !aligned(out, 2) ||
        !aligned(row_token, 4) || !aligned(offsets, 4) || !aligned(counts, 4))
        return MOEF_ERR_ALIGN;
    Gemm g{};
    g.a = u16(weight);
    g.b = u16(x);
    g.M = M;
    g.N = static_cast<int>(P);
    g.K = K;
    g.gated = gated;
    g.bias = u16(bias);
    g.out = out;
    g.act = static_cast<int>(act);
    g.E = E;
    g.offsets = offsets;
    g.counts = counts;
    g.row_token = row_token;
    g.b_rows = T;
    g.b_pitch = K;
    moef::BiasSum none = {};
    return run_gemm(g, &none, stream);
}

}  // namespace

extern "C" {

moef_status moe_linear(const void *x, const void *weight, const void *bias,
                       const void *residual, moef_activation act, void *out,
                       moef_out_type out_type, void *preact, int T, int N, int K,
                       cudaStream_t stream) {
    if (T < 0 || !valid_features(N) || !valid_features(K)) return MOEF_ERR_SHAPE;
    if (!valid_act(act) || (out_type != MOEF_OUT_BF16 && out_type != MOEF_OUT_FP32))
        return MOEF_ERR_ARG;
    if (T == 0) return MOEF_OK;
    if (!x || !weight || !out) return MOEF_ERR_NULL;
    if (!aligned(x, 2) || !aligned(weight, 2) || !aligned(bias, 2) || !aligned(residual, 2) ||
        !aligned(preact, 2) || !aligned(out, out_type == MOEF_OUT_FP32 ? 4 : 2))
        return MOEF_ERR_ALIGN;
    Gemm g{};
    g.a = u16(weight);
    g.b = u16(x);
    g.M = N;
    g.N = T;
    g.K = K;
    g.bias = u16(bias);
    g.residual = u16(residual);
    g.out = out;
    g.out_f32 = out_type == MOEF_OUT_FP32;
    g.preact = static_cast<uint16_t *>(preact);
    g.act = static_cast<int>(act);
    g.b_rows = T;
    g.b_pitch = K;
    moef::BiasSum none = {};
    return run_gemm(g, &none, stream);
}

size_t moe_linear_backward_workspace_bytes(int T, int N) {
    if (T < 0 || !valid_features(N)) return 0;
    return backward_bytes(T, N);
}

moef_status moe_linear_backward(const void *dout, const void *x, const void *weight,
                                moef_activation act, const void *preact,
                                void *dx, void *dweight, void *dbias, int T, int N, int K,
                                void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    return backward(dout, x, weight, act, preact, 0, dx, dweight, dbias, T, N, K, workspace,
                    workspace_bytes, stream);
}

moef_status moe_gated_ffn(const void *x, const void *weight, const void *bias,
                          moef_activation act, void *out, void *preact,
                          int T, int I, int H, cudaStream_t stream) {
    if (T < 0 || !valid_features(I) || !valid_features(H)) return MOEF_ERR_SHAPE;
    if (!valid_act(act)) return MOEF_ERR_ARG;
    if (T == 0) return MOEF_OK;
    if (!x || !weight || !out) return MOEF_ERR_NULL;
    if (!aligned(x, 2) || !aligned(weight, 2) || !aligned(bias, 2) || !aligned(preact, 2) ||
        !aligned(out, 2))
        return MOEF_ERR_ALIGN;
    Gemm g{};
    g.a = u16(weight);
    g.b = u16(x);
    g.M = I;
    g.N = T;
    g.K = H;
    g.gated = 1;
    g.bias = u16(bias);
    g.out = out;
    g.preact = static_cast<uint16_t *>(preact);
    g.act = static_cast<int>(act);
    g.b_rows = T;
    g.b_pitch = H;
    moef::BiasSum none = {};
    return run_gemm(g, &none, stream);
}

size_t moe_gated_ffn_backward_workspace_bytes(int T, int I) {
    if (T < 0 || !valid_features(I)) return 0;
    return backward_bytes(T, 2 * static_cast<int64_t>(I));
}

moef_status moe_gated_ffn_backward(const void *dout, const void *x, const void *weight,
                                   moef_activation act, const void *preact,
                                   void *dx, void *dweight, void *dbias, int T, int I, int H,
                                   void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
    return backward(dout, x, weight, act, preact, 1, dx, dweight, dbias, T, I, H, workspace,
                    workspace_bytes, stream);
}

int64_t moe_permute_rows(int T, int K, int E, int tile) {
    if (T < 0 || K < 1 || K > MOEF_MAX_K || E < 1 || E > MOEF_MAX_EXPERTS || tile < 1) return 0;
    const int64_t n = static_cast<int64_t>(T) * K;
    const int64_t used = n < E ? n : E;
    const int64_t rows = (n + used * (tile - 1)) / tile * tile;
    return rows > INT_MAX ? 0 : rows;
}

size_t moe_permute_workspace_bytes(int T, int K, int E) {
    if (T < 0 || K < 1 || K > MOEF_MAX_K || E < 1 || E > MOEF_MAX_EXPERTS) return 0;
    return static_cast<size_t>(moef::permute_chunks(static_cast<int64_t>(T) * K)) * E * 4;
}

moef_status moe_permute(const int32_t *expert_ids, int T, int K, int E, int tile,
                        int32_t *idx_map, int32_t *row_token, int64_t P,
                        int32_t *offsets, int32_t *counts,
                        void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (T < 0 || K < 1 || K > MOEF_MAX_K || E < 1 || E > MOEF_MAX_EXPERTS || tile < 1)
        return MOEF_ERR_SHAPE;
    const int64_t rows = moe_permute_rows(T, K, E, tile);
    if ((T > 0 && rows == 0) || P < rows || P > INT_MAX) return MOEF_ERR_SHAPE;
    const size_t need = moe_permute_workspace_bytes(T, K, E);
    if (!offsets || !counts || (need > 0 && !workspace) || (T > 0 && (!expert_ids || !idx_map)) ||
        (P > 0 && !row_token))
        return MOEF_ERR_NULL;
    if (workspace_bytes < need) return MOEF_ERR_SHAPE;
    if (!aligned(workspace, 16) || !aligned(expert_ids, 4) || !aligned(idx_map, 4) ||
        !aligned(row_token, 4) || !aligned(offsets, 4) || !aligned(counts, 4))
        return MOEF_ERR_ALIGN;
    return cuda_status(moef::launch_permute(expert_ids, T, K, E, tile, idx_map, row_token, P,
                                            offsets, counts, static_cast<int32_t *>(workspace),
                                            stream));
}

moef_status moe_expert_gated_ffn(const void *x, int64_t T, const int32_t *row_token,
                                 const int32_t *offsets, const int32_t *counts,
                                 const void *weight, const void *bias, moef_activation act,
                                 void *out, int64_t P, int E, int I, int H,
                                 cudaStream_t stream) {
    return expert_product(x, T, row_token, offsets, counts, weight, bias, act, 1, out, P, E, I,
                          H, stream);
}

moef_status moe_expert_linear(const void *x, int64_t T, const int32_t *row_token,
                              const int32_t *offsets, const int32_t *counts,
                              const void *weight, const void *bias, moef_activation act,
                              void *out, int64_t P, int E, int N, int K,
                              cudaStream_t stream) {
    return expert_product(x, T, row_token, offsets, counts, weight, bias, act, 0, out, P, E, N,
                          K, stream);
}

moef_status moe_ffn_lost_waits(unsigned *count) {
    if (!count) return MOEF_ERR_NULL;
    return cuda_status(moef::read_lost_waits(count));
}

}  // extern "C"
