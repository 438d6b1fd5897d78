// dz of the backward passes and its column sums.
//
//   linear  dz = dout * act'(preact)
//   gated   dz[:, i] = dout * u * act'(g),  dz[:, n + i] = dout * act(g)
//
// One pass over dout and preact (read once, dz written once): bound by HBM
// bandwidth.  A CTA takes sum_rows(T) rows of up to 32 vectors of columns, each
// warp one row at a time, or several where the columns do not fill it, all of a
// thread's loads of four steps in flight before their first use; the activation
// is a template argument, so its arithmetic overlaps.  dz is rounded to bf16, the
// operand type of the tensor cores, for both products: dx and dweight are then off
// by 2.35e-3 (root mean square, relative), where their own rounding alone is
// 1.66e-3.  The column sums build up in registers, in fp32 and before dz is
// rounded; the CTA adds its lanes' sums in order and writes one row of `partial`,
// whose rows are then added in order (no atomics: equal calls give equal bits) by
// idle warps of the product that follows, or by a kernel of its own.  2040 x 4096
// with GELU takes 12.2 us (4.1 TB/s; with the activation chosen per value and 32
// rows a thread it took 40 us), 4096 x 2048 gated with SiLU 15.8 us (5.3 TB/s).
#include "ffn.cuh"
#include "tc.cuh"
#include "vec.cuh"

namespace moef {
namespace {

constexpr int kDzWarps = 8;
constexpr int kDzThreads = 32 * kDzWarps;
constexpr int kDzRows = 4;              // of a thread at a time
constexpr int kMinRows = kDzWarps * kDzRows, kMaxSums = 512;

template <int VEC, bool GATED, int ACT>
__global__ void __launch_bounds__(kDzThreads)
dz_kernel(const uint16_t *dout, const uint16_t *preact, uint16_t *dz, int64_t pitch,
          float *partial, int T, int n, int rows, int log_lanes) {
    using Ops = VecOps<VEC>;
    using V = typename Ops::V;
    constexpr int kHalves = GATED ? 2 : 1;
    __shared__ float sums[kDzWarps][kHalves][32 * VEC];
    // 2^log_lanes lanes of a warp along the columns, the rest along the rows
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int across = VEC << log_lanes, at_once = 32 >> log_lanes;
    const int cols = kHalves * n;
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * rows;
    const int64_t end = begin + rows < T ? begin + rows : T;
    const int64_t first = begin + warp * at_once + (lane >> log_lanes);
    wait_previous_kernel();
    allow_next_kernel();
    for (int i0 = blockIdx.y * across; i0 < n; i0 += gridDim.y * across) {
        const int i = i0 + (lane & ((1 << log_lanes) - 1)) * VEC;
        float sum[kHalves][VEC] = {};
        for (int64_t t0 = first; i < n && t0 < end; t0 += kMinRows * at_once) {
            V d[kDzRows] = {}, z[kHalves][kDzRows] = {};
#pragma unroll
            for (int r = 0; r < kDzRows; ++r) {
                const int64_t t = t0 + r * kDzWarps * at_once;
                if (t < end) {
                    d[r] = Ops::load(dout + t * n + i);
                    if (GATED || ACT != MOEF_ACT_NONE) z[0][r] = Ops::load(preact + t * cols + i);
                    if constexpr (GATED) z[1][r] = Ops::load(preact + t * cols + n + i);
                }
            }
#pragma unroll
            for (int r = 0; r < kDzRows; ++r) {
                const int64_t t = t0 + r * kDzWarps * at_once;
                if (t >= end) break;
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
            for (int c = threadIdx.x; c < kHalves * across; c += kDzThreads) {
                const int h = c >= across, k = c - h * across;
                float v = 0.f;
                for (int j = 0; j < at_once; ++j)
#pragma unroll
                    for (int w = 0; w < kDzWarps; ++w) v += sums[w][h][j * across + k];
                if (i0 + k < n)
                    partial[static_cast<int64_t>(blockIdx.x) * cols + h * n + i0 + k] = v;
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
    const int rows = sum_rows(T);
    int log_lanes = 0;
    while (log_lanes < 5 && VEC << log_lanes < n) ++log_lanes;
    const int across = (n - 1) / (VEC << log_lanes) + 1;
    const dim3 grid(static_cast<unsigned>((T - 1) / rows + 1),
                    static_cast<unsigned>(across < 65535 ? across : 65535));
    auto go = [&](auto *kernel) {
        return start(kernel, grid, kDzThreads, stream, dout, preact, dz, pitch, partial, T, n,
                     rows, log_lanes);
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

// A step of a CTA's warps, and so many steps that at most kMaxSums rows of sums
// are left to add, which takes one thread a column.
int sum_rows(int T) {
    int64_t rows = kMinRows;
    while ((T - 1) / rows >= kMaxSums) rows *= 2;
    return static_cast<int>(rows);
}

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
