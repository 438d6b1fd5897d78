// dz of the backward passes and its column sums.
//
//   linear  dz = dout * act'(preact)
//   gated   dz[:, i] = dout * u * act'(g),  dz[:, n + i] = dout * act(g)
//
// One pass over dout and preact (read once, dz written once): bound by HBM
// bandwidth.  A thread owns one vector of columns and walks kBiasRows rows of
// it, so the column sums build up in its registers, in fp32 and before dz is
// rounded; each CTA writes its rows' sums as one row of `partial`, and a
// second kernel adds those rows in a fixed order (no atomics: equal calls
// give equal bits).
#include "ffn.cuh"
#include "vec.cuh"

namespace moef {
namespace {

constexpr int kDzThreads = 128;

template <int VEC, bool GATED>
__global__ void __launch_bounds__(kDzThreads)
dz_kernel(const uint16_t *dout, const uint16_t *preact, int act, uint16_t *dz, float *partial,
          int T, int n) {
    using Ops = VecOps<VEC>;
    const int cols = GATED ? 2 * n : n;
    const int t0 = blockIdx.x * kBiasRows, t1 = min(T - t0, kBiasRows) + t0;
    for (int i = (blockIdx.y * kDzThreads + threadIdx.x) * VEC; i < n;
         i += gridDim.y * kDzThreads * VEC) {
        float sum[GATED ? 2 : 1][VEC] = {};
#pragma unroll 4
        for (int t = t0; t < t1; ++t) {
            const int64_t row = static_cast<int64_t>(t) * cols + i;
            float d[VEC], g[VEC], r[VEC];
            Ops::to_f32(Ops::load(dout + static_cast<int64_t>(t) * n + i), d);
            if constexpr (GATED) {
                float u[VEC], r2[VEC];
                Ops::to_f32(Ops::load(preact + row), g);
                Ops::to_f32(Ops::load(preact + row + n), u);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    float a;
                    const float da = act_grad(g[j], act, &a);
                    r[j] = d[j] * u[j] * da;
                    r2[j] = d[j] * a;
                    sum[0][j] += r[j];
                    sum[1][j] += r2[j];
                }
                // read again by both products: kept in L2 where it fits
                *reinterpret_cast<typename Ops::V *>(dz + row) = Ops::from_f32(r);
                *reinterpret_cast<typename Ops::V *>(dz + row + n) = Ops::from_f32(r2);
            } else {
                if (preact) Ops::to_f32(Ops::load(preact + row), g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    float a;
                    r[j] = preact ? d[j] * act_grad(g[j], act, &a) : d[j];
                    sum[0][j] += r[j];
                }
                if (dz) *reinterpret_cast<typename Ops::V *>(dz + row) = Ops::from_f32(r);
            }
        }
        if (partial) {
#pragma unroll
            for (int h = 0; h < (GATED ? 2 : 1); ++h)
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    partial[static_cast<int64_t>(blockIdx.x) * cols + h * n + i + j] = sum[h][j];
        }
    }
}

// dbias[c] = sum of partial[:, c]: 32 columns a CTA, 8 warps taking every
// eighth row, their sums added in warp order.
__global__ void __launch_bounds__(256)
bias_sum_kernel(const float *partial, int rows, int cols, uint16_t *dbias) {
    __shared__ float s[8][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x / 32;
    float sum = 0.f;
    if (c < cols)
        for (int r = w; r < rows; r += 8) sum += partial[static_cast<int64_t>(r) * cols + c];
    s[w][threadIdx.x & 31] = sum;
    __syncthreads();
    if (w == 0 && c < cols) {
        sum = s[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < 8; ++k) sum += s[k][threadIdx.x];
        dbias[c] = __bfloat16_as_ushort(__float2bfloat16_rn(sum));
    }
}

template <int VEC>
void start_dz(const uint16_t *dout, const uint16_t *preact, int act, int gated, uint16_t *dz,
              float *partial, int T, int n, cudaStream_t stream) {
    const int64_t across = (static_cast<int64_t>(n) + kDzThreads * VEC - 1) / (kDzThreads * VEC);
    const dim3 grid(static_cast<unsigned>((T - 1) / kBiasRows + 1),
                    static_cast<unsigned>(across < 65535 ? across : 65535));
    if (gated)
        dz_kernel<VEC, true><<<grid, kDzThreads, 0, stream>>>(dout, preact, act, dz, partial, T, n);
    else
        dz_kernel<VEC, false><<<grid, kDzThreads, 0, stream>>>(dout, preact, act, dz, partial, T, n);
}

}  // namespace

cudaError_t launch_dz(const uint16_t *dout, const uint16_t *preact, int act, int gated,
                      uint16_t *dz, float *partial, uint16_t *dbias, int T, int n,
                      cudaStream_t stream) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(dout) | reinterpret_cast<uintptr_t>(preact) |
                           reinterpret_cast<uintptr_t>(dz);
    float *part = dbias ? partial : nullptr;
    if (n % 8 == 0 && bits % 16 == 0)
        start_dz<8>(dout, preact, act, gated, dz, part, T, n, stream);
    else
        start_dz<1>(dout, preact, act, gated, dz, part, T, n, stream);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || !dbias) return err;
    const int cols = gated ? 2 * n : n;
    bias_sum_kernel<<<(cols + 31) / 32, 256, 0, stream>>>(partial, (T - 1) / kBiasRows + 1,
                                                          cols, dbias);
    return cudaGetLastError();
}

}  // namespace moef
