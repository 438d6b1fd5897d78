// dz of the backward passes and its column sums.
//
//   linear  dz = dout * act'(preact)
//   gated   dz[:, i] = dout * u * act'(g),  dz[:, n + i] = dout * act(g)
//
// One pass over dout and preact (read once, dz written once): bound by HBM
// bandwidth.  A CTA takes kBiasRows rows of 32 vectors of columns, a warp
// every eighth row, all of a thread's loads in flight before their first use;
// the activation is a template argument, so its arithmetic overlaps.  The
// column sums build up in registers, in fp32 and before dz is rounded; the
// CTA adds its warps' sums in order and writes one row of `partial`, whose rows
// are then added in order (no atomics: equal calls give equal bits) by idle
// warps of the product that follows, or by a kernel of its own.  2040 x 4096 with
// GELU takes 12.6 us (4.0 TB/s; with the activation chosen per value and 32 rows
// a thread it took 40 us), 4096 x 2048 gated with SiLU 15.5 us (5.4 TB/s).
#include "ffn.cuh"
#include "tc.cuh"
#include "vec.cuh"

namespace moef {
namespace {

constexpr int kDzWarps = 8;
constexpr int kDzThreads = 32 * kDzWarps;
constexpr int kDzRows = kBiasRows / kDzWarps;       // rows per thread

template <int VEC, bool GATED, int ACT>
__global__ void __launch_bounds__(kDzThreads)
dz_kernel(const uint16_t *dout, const uint16_t *preact, uint16_t *dz, int64_t pitch,
          float *partial, int T, int n) {
    using Ops = VecOps<VEC>;
    using V = typename Ops::V;
    constexpr int kHalves = GATED ? 2 : 1;
    __shared__ float sums[kDzWarps][kHalves][32 * VEC];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int cols = kHalves * n;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kBiasRows;
    wait_previous_kernel();
    allow_next_kernel();
    for (int i0 = blockIdx.y * 32 * VEC; i0 < n; i0 += gridDim.y * 32 * VEC) {
        const int i = i0 + lane * VEC;
        float sum[kHalves][VEC] = {};
        if (i < n) {
            V d[kDzRows] = {}, z[kHalves][kDzRows] = {};
#pragma unroll
            for (int r = 0; r < kDzRows; ++r) {
                const int64_t t = t0 + warp + r * kDzWarps;
                if (t < T) {
                    d[r] = Ops::load(dout + t * n + i);
                    if (GATED || ACT != MOEF_ACT_NONE) z[0][r] = Ops::load(preact + t * cols + i);
                    if constexpr (GATED) z[1][r] = Ops::load(preact + t * cols + n + i);
                }
            }
#pragma unroll
            for (int r = 0; r < kDzRows; ++r) {
                const int64_t t = t0 + warp + r * kDzWarps;
                if (t >= T) break;
                float dv[VEC], gv[VEC], out[kHalves][VEC];
                Ops::to_f32(d[r], dv);
                Ops::to_f32(z[0][r], gv);
                if constexpr (GATED) {
                    float uv[VEC];
                    Ops::to_f32(z[1][r], uv);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        float a;
                        const float da = act_grad(gv[j], ACT, &a);
                        out[0][j] = dv[j] * uv[j] * da;
                        out[1][j] = dv[j] * a;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        float a;
                        out[0][j] = ACT == MOEF_ACT_NONE ? dv[j]
                                                         : dv[j] * act_grad(gv[j], ACT, &a);
                    }
                }
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) sum[h][j] += out[h][j];
                    // read again by both products: an ordinary store keeps it in L2
                    if (dz) *reinterpret_cast<V *>(dz + t * pitch + h * n + i) =
                                Ops::from_f32(out[h]);
                }
            }
        }
        if (partial) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int j = 0; j < VEC; ++j) sums[warp][h][lane * VEC + j] = sum[h][j];
            __syncthreads();
            for (int c = threadIdx.x; c < kHalves * 32 * VEC; c += kDzThreads) {
                const int h = c / (32 * VEC), k = c % (32 * VEC);
                float v = sums[0][h][k];
#pragma unroll
                for (int w = 1; w < kDzWarps; ++w) v += sums[w][h][k];
                if (i0 + k < n) partial[blockIdx.x * static_cast<int64_t>(cols) + h * n + i0 + k] = v;
            }
            __syncthreads();
        }
    }
}

__global__ void __launch_bounds__(32)
bias_sum_kernel(const BiasSum b) {
    wait_previous_kernel();
    allow_next_kernel();
    sum_columns(b, blockIdx.x * 32 + threadIdx.x);
}

template <typename... Params, typename... Args>
cudaError_t start(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t stream,
                  Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

template <int VEC, bool GATED>
cudaError_t start_dz(const uint16_t *dout, const uint16_t *preact, int act, uint16_t *dz,
                     int64_t pitch, float *partial, int T, int n, cudaStream_t stream) {
    const int64_t across = (static_cast<int64_t>(n) + 32 * VEC - 1) / (32 * VEC);
    const dim3 grid(static_cast<unsigned>((T - 1) / kBiasRows + 1),
                    static_cast<unsigned>(across < 65535 ? across : 65535));
    auto go = [&](auto *kernel) {
        return start(kernel, grid, kDzThreads, stream, dout, preact, dz, pitch, partial, T, n);
    };
    switch (act) {
        case MOEF_ACT_SILU: return go(dz_kernel<VEC, GATED, MOEF_ACT_SILU>);
        case MOEF_ACT_GELU: return go(dz_kernel<VEC, GATED, MOEF_ACT_GELU>);
        case MOEF_ACT_GELU_TANH: return go(dz_kernel<VEC, GATED, MOEF_ACT_GELU_TANH>);
        case MOEF_ACT_RELU: return go(dz_kernel<VEC, GATED, MOEF_ACT_RELU>);
        default: return go(dz_kernel<VEC, GATED, MOEF_ACT_NONE>);
    }
}

}  // namespace

cudaError_t launch_dz(const uint16_t *dout, const uint16_t *preact, int act, int gated,
                      uint16_t *dz, int64_t pitch, float *partial, int T, int n,
                      cudaStream_t stream) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(dout) | reinterpret_cast<uintptr_t>(preact) |
                           reinterpret_cast<uintptr_t>(dz);
    const bool vec = n % 8 == 0 && bits % 16 == 0;
    if (gated)
        return vec ? start_dz<8, true>(dout, preact, act, dz, pitch, partial, T, n, stream)
                   : start_dz<1, true>(dout, preact, act, dz, pitch, partial, T, n, stream);
    return vec ? start_dz<8, false>(dout, preact, act, dz, pitch, partial, T, n, stream)
               : start_dz<1, false>(dout, preact, act, dz, pitch, partial, T, n, stream);
}

cudaError_t launch_bias_sum(const BiasSum &b, cudaStream_t stream) {
    if (!b.dbias) return cudaSuccess;
    return start(bias_sum_kernel, dim3(static_cast<unsigned>((b.cols + 31) / 32)), 32, stream, b);
}

}  // namespace moef
