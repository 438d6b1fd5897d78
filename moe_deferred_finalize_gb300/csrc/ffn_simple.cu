// The plain form of the products of moe_ffn.h: a tiled kernel of fp32
// multiply-adds over operands of any size, alignment and orientation.  It
// serves what the tensor-core kernels cannot (their copies need 16-byte
// aligned rows): odd feature counts and misaligned views.
//
// Out tile 64 (m) x 64 (n) per CTA of 256 threads, 4 x 4 outputs a thread
// (8 x 4 in the gated form: gate and up rows), k in steps of 16 through
// shared memory.
#include "ffn.cuh"
#include "vec.cuh"

namespace moef {
namespace {

constexpr int kTile = 64, kStep = 16, kSimpleThreads = 256;

__device__ __forceinline__ float bf16_at(const uint16_t *p, int64_t i) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(p + i)) << 16);
}

__device__ __forceinline__ uint16_t to_bf16(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// One operand tile into shared memory as fp32: rows r0 .. r0 + 64 (row(i) in
// memory, negative: zeros), k0 .. k0 + 16.  The threads run along the
// operand's contiguous axis.
template <typename Row>
__device__ __forceinline__ void load_tile(float (*s)[kTile + 1], const uint16_t *p, int mn,
                                          int64_t pitch, int k0, int K, Row row) {
    for (int i = threadIdx.x; i < kTile * kStep; i += kSimpleThreads) {
        const int r = mn ? i % kTile : i / kStep;
        const int k = mn ? i / kTile : i % kStep;
        const int64_t at = row(r);
        float v = 0.f;
        if (at >= 0 && k0 + k < K)
            v = bf16_at(p, mn ? static_cast<int64_t>(k0 + k) * pitch + at
                              : at * pitch + k0 + k);
        s[k][r] = v;
    }
}

template <bool GATED>
__global__ void __launch_bounds__(kSimpleThreads)
gemm_simple_kernel(const Gemm g) {
    __shared__ float sa[GATED ? 2 : 1][kStep][kTile + 1];
    __shared__ float sb[kStep][kTile + 1];
    const int e = blockIdx.z;
    const int m0 = blockIdx.x * kTile;
    int64_t first = 0;
    int64_t count = g.N;
    if (g.E) {
        first = g.offsets[e];
        count = min(static_cast<int64_t>(g.counts[e]), static_cast<int64_t>(g.N) - first);
        if (first < 0) return;
    }
    const int arows = GATED ? 2 * g.M : g.M;
    const uint16_t *a = g.a + static_cast<int64_t>(e) * arows * g.K;
    const uint16_t *bias = g.bias ? g.bias + static_cast<int64_t>(e) * arows : nullptr;
    const int64_t a_pitch = g.a_mn ? arows : g.K;
    const int64_t b_pitch = g.b_pitch;
    const int tm = threadIdx.x % 16, tn = threadIdx.x / 16;

    for (int64_t n0 = static_cast<int64_t>(blockIdx.y) * kTile; n0 < count;
         n0 += static_cast<int64_t>(gridDim.y) * kTile) {
        float acc[GATED ? 2 : 1][4][4] = {};
        for (int k0 = 0; k0 < g.K; k0 += kStep) {
#pragma unroll
            for (int h = 0; h < (GATED ? 2 : 1); ++h)
                load_tile(sa[h], a, g.a_mn, a_pitch, k0, g.K, [&](int r) -> int64_t {
                    return m0 + r < g.M ? static_cast<int64_t>(h) * g.M + m0 + r : -1;
                });
            load_tile(sb, g.b, g.b_mn, b_pitch, k0, g.K, [&](int r) -> int64_t {
                if (n0 + r >= count) return -1;
                int64_t row = first + n0 + r;
                if (g.row_token) row = __ldg(g.row_token + row);
                return row < g.b_rows ? row : -1;
            });
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kStep; ++k) {
                float fb[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) fb[j] = sb[k][tn * 4 + j];
#pragma unroll
                for (int h = 0; h < (GATED ? 2 : 1); ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float fa = sa[h][k][tm + 16 * i];
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[h][i][j] = fmaf(fa, fb[j], acc[h][i][j]);
                    }
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (n0 + tn * 4 + j >= count) break;
            const int64_t n = first + n0 + tn * 4 + j;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = m0 + tm + 16 * i;
                if (m >= g.M) break;
                float z = acc[0][i][j];
                if (bias) z += bf16_at(bias, m);
                float v;
                if constexpr (GATED) {
                    float u = acc[1][i][j];
                    if (bias) u += bf16_at(bias, g.M + m);
                    if (g.preact) {
                        g.preact[n * 2 * g.M + m] = to_bf16(z);
                        g.preact[n * 2 * g.M + g.M + m] = to_bf16(u);
                    }
                    v = act_value(z, g.act) * u;
                } else {
                    if (g.preact) g.preact[n * g.M + m] = to_bf16(z);
                    v = act_value(z, g.act);
                    if (g.residual) v += bf16_at(g.residual, n * g.M + m);
                }
                if (g.out_f32) static_cast<float *>(g.out)[n * g.M + m] = v;
                else static_cast<uint16_t *>(g.out)[n * g.M + m] = to_bf16(v);
            }
        }
    }
}

}  // namespace

cudaError_t launch_gemm_simple(const Gemm &g, cudaStream_t stream) {
    const int64_t m_tiles = (static_cast<int64_t>(g.M) + kTile - 1) / kTile;
    const int64_t n_tiles = (static_cast<int64_t>(g.N) + kTile - 1) / kTile;
    const int64_t experts = g.E ? g.E : 1;
    const dim3 grid(static_cast<unsigned>(m_tiles),
                    static_cast<unsigned>(g.E ? (n_tiles < 8 ? n_tiles : 8)
                                              : (n_tiles < 65535 ? n_tiles : 65535)),
                    static_cast<unsigned>(experts));
    if (g.gated) gemm_simple_kernel<true><<<grid, kSimpleThreads, 0, stream>>>(g);
    else gemm_simple_kernel<false><<<grid, kSimpleThreads, 0, stream>>>(g);
    return cudaGetLastError();
}

}  // namespace moef
