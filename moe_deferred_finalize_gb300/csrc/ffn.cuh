// Declarations shared by the translation units of the matrix products around
// the finalize (moe_ffn.h): the description of one product, the activations
// and the launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_ffn.h"

namespace moef {

// One product out[n, m] = epilogue(sum_k A[m, k] B[n, k]), m along the
// output's rows (contiguous), so the three products of a layer read their
// operands as they lie:
//   forward   A = weight [M, K],   B = x [N, K]         (both k-contiguous)
//   dx        A = weight [K, M],   B = dz [N, K]        (A m-contiguous)
//   dweight   A = x [K, M],        B = dz [K, N]        (both transposed)
// Gated: A has 2M rows, the gate rows then the up rows, and
// out = act(gate) * up.  Grouped (E > 0): A is [E, M or 2M, K] ([E, K, M] when m is
// contiguous), the rows n of expert e are offsets[e] .. offsets[e] + counts[e], row n
// read from row row_token[n] of B.
// Grouped dweight: k runs over each expert's rows of A = x [K, M] and B = dz [K, N],
// both in the layout, out [E, N, M].
struct Gemm {
    const uint16_t *a, *b;
    int a_mn, b_mn;             // 1: the operand is contiguous along m (n), not k
    int M, N, K;
    int gated;
    const uint16_t *bias;       // [M] or [2M] (per expert), or null
    const uint16_t *residual;   // bf16 [N, M] or null
    void *out;                  // [N, M]
    int out_f32;
    uint16_t *preact;           // bf16 [N, M] or [N, 2M], or null
    int act;
    int E;                      // 0: not grouped
    const int32_t *offsets, *counts, *row_token;
    int64_t b_rows;             // rows of B
    int64_t b_pitch;            // values from one of its rows (of k: b_mn) to the next
    int64_t a_pitch;            // the same of A, for grouped dweight
    int a_zeros, b_zeros;       // the operand has zeros behind spaced rows
};

// Steps of `step` values that cover k >= 1 of them.  k is a token count in
// dweight, up to 2^31 - 1, which rounding up in 32 bits would pass.
__host__ __device__ constexpr int steps_of(int k, int step) { return (k - 1) / step + 1; }
static_assert(steps_of(INT32_MAX, 64) == 1 << 25 && steps_of(64, 64) == 1 && steps_of(65, 64) == 2,
              "steps of the longest sums");

// Tiled kernel of single-value loads: any size, alignment and layout.
cudaError_t launch_gemm_simple(const Gemm &g, cudaStream_t stream);

// The column sums that launch_dz left per sum_rows(T) rows: dbias[c] = sum of
// partial[:, c], rows added in order.
struct BiasSum {
    const float *partial;       // fp32 [rows, cols]
    uint16_t *dbias;            // bf16 [cols], null: nothing to do
    int rows, cols;
};
cudaError_t launch_bias_sum(const BiasSum &b, cudaStream_t stream);

// The tensor-core kernels.  False (nothing launched) when an operand's
// alignment or pitch rules them out; otherwise *err is the launch's result.
// The launch also does `bias` on warps that have nothing to copy.
bool launch_gemm_tc(const Gemm &g, const BiasSum &bias, int num_sms, cudaStream_t stream,
                    cudaError_t *err);

// Two products (not grouped, not gated) in one launch; false (nothing launched)
// also when two launches are priced lower.
bool launch_two_gemms_tc(const Gemm *g, const BiasSum &bias, int num_sms, cudaStream_t stream,
                         cudaError_t *err);

// The grouped dweight, on the tensor cores: both operands 16-byte aligned, pitches
// multiples of 8.
cudaError_t launch_group_dweight(const Gemm &g, int num_sms, cudaStream_t stream);

// The kernel for a handful of rows; false (nothing launched) when the sizes or
// alignment are not its own, or the tensor-core one is faster.
constexpr int kDecodeRows = 8;
bool launch_gemm_decode(const Gemm &g, int num_sms, cudaStream_t stream, cudaError_t *err);

// Barrier waits that gave up since the library was loaded on this device.
cudaError_t read_lost_waits(unsigned *count);

// dz of the backward passes, its bf16 rounding into dz [T, pitch] (null: none;
// the values past cols are not written), and its column sums over sum_rows(T)
// rows at a time into partial (fp32 [ceil(T / sum_rows(T)), cols], null: none).
// Linear: cols = n, dz = dout * act'(preact), or dout without preact.  Gated:
// cols = 2n, dout [T, n], preact [T, 2n].
int sum_rows(int T);        // T >= 1
cudaError_t launch_dz(const uint16_t *dout, const uint16_t *preact, int act, int gated,
                      uint16_t *dz, int64_t pitch, float *partial, int T, int n,
                      cudaStream_t stream);

// The grouped layout (moe_permute).  permute_chunks: rows of E counts that
// the workspace holds for that many slots (0: none needed).
int permute_chunks(int64_t slots);
cudaError_t launch_permute(const int32_t *ids, int T, int K, int E, int tile, int32_t *idx_map,
                           int32_t *row_token, int64_t P, int32_t *offsets, int32_t *counts,
                           int32_t *workspace, cudaStream_t stream);

#ifdef __CUDACC__
namespace {

// Whether an expert's rows, rounded up to a multiple of 16, end before the next
// expert's first row (or the end of the layout) and the buffer's end.  When all do,
// no two experts share the rows in between: the backward pass fills those of its
// workspace with zeros, and its product may read them.  Both ask this.
__device__ __forceinline__ int spaced_rows(int first, int rows, int next, int64_t P) {
    const int64_t end = static_cast<int64_t>(first) + ((static_cast<int64_t>(rows) + 15) & ~15LL);
    return first >= 0 && first <= next && end <= next && end <= P;
}

// 2^x and 1 / x as one instruction each, results below the normal range as 0,
// which the activations multiply into an error below 1e-35.  (__expf and
// __fdividef spend three or four instructions more on that range; the issue of
// instructions is what activations cost: 20 million SiLUs 6 us, now 5.)
__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_ftz(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.44269504f;

// 1 / (1 + exp(-z)).
__device__ __forceinline__ float sigmoid(float z) {
    return reciprocal_ftz(1.f + exp2_ftz(-kLog2e * z));
}

// sigmoid(2 sqrt(2/pi) (z + 0.044715 z^3)): (1 + tanh) / 2 of GELU's tanh form.
__device__ __forceinline__ float sigmoid_cubic(float z) {
    const float c = -1.59576912f * kLog2e;
    return reciprocal_ftz(1.f + exp2_ftz(z * (c + 0.044715f * c * (z * z))));
}

// Phi(z), the standard normal distribution function, and exp(-z^2 / 2) in *bell.
// Phi(-u) exp(u^2 / 2) is smooth and bounded on u >= 0; a polynomial of degree 7 in
// t = 1 / (1 + 0.35 u) takes its place, fitted for the least relative error on
// u <= 14: with these coefficients it alternates nine times between -3.4e-7 (u =
// 0.10, 1.04, 3.61, 9.33) and 2.8e-7 (u = 0, 0.43, 2.03, 6.0, 12.8).  The upper half
// is 1 - Phi(-u).  The exponential's argument carries three roundings, so that the
// error of Phi grows with z^2: at most (0.75 z^2 + 15) 2^-23 of its size, and by an
// emulation 1e-6 down to z = -4, 4e-6 to -9, 8e-6 where Phi passes 1e-30 (-11.5).
// 20 million GELUs in a product's epilogue took 31 us with erfcf, 10 so.
__device__ __forceinline__ float normal_cdf(float z, float *bell) {
    const float t = reciprocal_ftz(1.f + 0.35f * fabsf(z));
    float q = 0.04894243553f;
    q = q * t - 0.2021192462f;
    q = q * t + 0.2406407595f;
    q = q * t - 0.01702339575f;
    q = q * t + 0.1559614688f;
    q = q * t + 0.1333550960f;
    q = q * t + 0.1402703375f;
    q = q * t - 2.731550558e-5f;
    *bell = exp2_ftz(-0.5f * kLog2e * (z * z));
    q *= *bell;
    return z < 0.f ? q : 1.f - q;
}

// The activations in the forms that lose nothing to cancellation: z sigmoid(q)
// stays accurate relative to its size where 1 + tanh or 1 + erf would cancel.
__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case MOEF_ACT_SILU: return z * sigmoid(z);
        case MOEF_ACT_GELU: {
            float bell;
            return z * normal_cdf(z, &bell);
        }
        case MOEF_ACT_GELU_TANH: return z * sigmoid_cubic(z);
        case MOEF_ACT_RELU: return z > 0.f || z != z ? z : 0.f;
        default: return z;
    }
}

// One column of a BiasSum.
__device__ __forceinline__ void sum_columns(const BiasSum &b, int c) {
    if (c >= b.cols) return;
    float sum = 0.f;
#pragma unroll 16
    for (int r = 0; r < b.rows; ++r) sum += b.partial[static_cast<int64_t>(r) * b.cols + c];
    b.dbias[c] = __bfloat16_as_ushort(__float2bfloat16_rn(sum));
}

// act'(z), and act(z) in *value.
__device__ __forceinline__ float act_grad(float z, int act, float *value) {
    switch (act) {
        case MOEF_ACT_SILU: {
            const float s = sigmoid(z);
            *value = z * s;
            return s * (1.f + z * (1.f - s));
        }
        case MOEF_ACT_GELU: {
            float bell;
            const float phi = normal_cdf(z, &bell);
            *value = z * phi;
            return phi + 0.39894228f * z * bell;
        }
        case MOEF_ACT_GELU_TANH: {
            const float s = sigmoid_cubic(z);
            *value = z * s;
            const float d = s * (1.f - s);      // 0 far out, where z * z may overflow
            return d == 0.f ? s : s + d * z * 1.59576912f * (1.f + 0.134145f * z * z);
        }
        case MOEF_ACT_RELU:
            *value = z > 0.f || z != z ? z : 0.f;
            return z > 0.f ? 1.f : 0.f;
        default: *value = z; return 1.f;
    }
}

}  // namespace
#endif

}  // namespace moef
