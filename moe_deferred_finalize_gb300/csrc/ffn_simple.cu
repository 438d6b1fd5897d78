// The products of moe_ffn.h over operands of any size, alignment and
// orientation: what the tensor-core kernels cannot take (their copies need
// 16-byte aligned rows), such as odd inner sizes and misaligned views.
//
// A CTA computes 128 rows of A (gated: 64 gate rows and their 64 up rows) by 64
// rows of B.  The threads load single bf16 values along the operand's
// contiguous axis, the next step's into registers while the current one is
// multiplied, and lay them k-contiguous into shared memory, where ldmatrix
// feeds mma.m16n8k16; eight warps own 32 x 32 outputs each.  Bound by the
// 2-byte loads and stores: 4096 x 4096 x 4095 takes 2.25 ms (61 TFLOP/s; with
// fp32 multiply-adds it took 7 ms).
#include "ffn.cuh"
#include "tc.cuh"
#include "vec.cuh"

namespace moef {
namespace {

constexpr int kRowsA = 128, kRowsB = 64, kStep = 32, kSimpleThreads = 256;
constexpr int kPad = kStep + 8;         // 80 bytes a row: ldmatrix rows in distinct banks

__device__ __forceinline__ float bf16_at(const uint16_t *p, int64_t i) {
    return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}

__device__ __forceinline__ uint16_t to_bf16(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// A step's values of one operand: ROWS rows of 32 k, in registers.
template <int ROWS>
struct Staged {
    uint16_t v[ROWS * kStep / kSimpleThreads];

    __device__ static __forceinline__ void place(int i, int mn, int *row, int *k) {
        const int at = threadIdx.x + i * kSimpleThreads;
        *row = mn ? at % ROWS : at / kStep;
        *k = mn ? at / ROWS : at % kStep;
    }
    // row_at(r): the operand's row (negative: zeros)
    template <typename Row>
    __device__ __forceinline__ void load(const uint16_t *p, int mn, int64_t pitch, int k0, int K,
                                         Row row_at) {
#pragma unroll
        for (int i = 0; i < ROWS * kStep / kSimpleThreads; ++i) {
            int r, k;
            place(i, mn, &r, &k);
            const int64_t row = row_at(r);
            v[i] = 0;
            if (row >= 0 && k0 + k < K)
                v[i] = mn ? p[static_cast<int64_t>(k0 + k) * pitch + row]
                          : p[row * pitch + k0 + k];
        }
    }
    __device__ __forceinline__ void store(uint16_t (*s)[kPad], int mn) const {
#pragma unroll
        for (int i = 0; i < ROWS * kStep / kSimpleThreads; ++i) {
            int r, k;
            place(i, mn, &r, &k);
            s[r][k] = v[i];
        }
    }
};

// Four 8 x 8 matrices, one row address per lane.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const uint16_t *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_addr(p)) : "memory");
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool GATED>
__global__ void __launch_bounds__(kSimpleThreads, 2)
gemm_simple_kernel(const Gemm g) {
    constexpr int kFeatures = GATED ? 64 : 128;
    __shared__ __align__(16) uint16_t sa[kRowsA][kPad], sb[kRowsB][kPad];
    const int e = blockIdx.z;
    const int m0 = blockIdx.x * kFeatures;
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
    const int steps = steps_of(g.K, kStep);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int wm = warp & 3, wn = warp >> 2;
    // the warp's two blocks of 16 rows of A: gate and up, or adjacent ones
    const int block0 = GATED ? wm * 16 : wm * 32, block1 = GATED ? 64 + wm * 16 : wm * 32 + 16;

    auto a_row = [&](int r) -> int64_t {
        const int m = m0 + (GATED ? r & 63 : r);
        return m < g.M ? (GATED && r >= 64 ? g.M + m : m) : -1;
    };
    for (int64_t n0 = static_cast<int64_t>(blockIdx.y) * kRowsB; n0 < count;
         n0 += static_cast<int64_t>(gridDim.y) * kRowsB) {
        auto b_row = [&](int r) -> int64_t {
            if (n0 + r >= count) return -1;
            int64_t row = first + n0 + r;
            if (g.row_token) row = g.row_token[row];
            return row < g.b_rows ? row : -1;
        };
        float acc[2][4][4] = {};
        Staged<kRowsA> next_a;
        Staged<kRowsB> next_b;
        next_a.load(a, g.a_mn, a_pitch, 0, g.K, a_row);
        next_b.load(g.b, g.b_mn, g.b_pitch, 0, g.K, b_row);
        for (int step = 0; step < steps; ++step) {
            next_a.store(sa, g.a_mn);
            next_b.store(sb, g.b_mn);
            __syncthreads();
            if (step + 1 < steps) {
                const int k0 = (step + 1) * kStep;
                next_a.load(a, g.a_mn, a_pitch, k0, g.K, a_row);
                next_b.load(g.b, g.b_mn, g.b_pitch, k0, g.K, b_row);
            }
#pragma unroll
            for (int k = 0; k < kStep; k += 16) {
                uint32_t fa[2][4], fb[2][4];
                const int row = lane & 15, half = lane >> 4;
                ldmatrix4(fa[0], &sa[block0 + row][k + 8 * half]);
                ldmatrix4(fa[1], &sa[block1 + row][k + 8 * half]);
                // b: n rows 0..7, 8..15, each k 0..7 and 8..15
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    ldmatrix4(fb[j], &sb[wn * 32 + j * 16 + (lane & 7) + 8 * half]
                                        [k + (lane & 8)]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma(acc[i][j], fa[i], fb[j >> 1][(j & 1) * 2], fb[j >> 1][(j & 1) * 2 + 1]);
            }
            __syncthreads();
        }
        auto finish = [&](int m, int c, float z, float u) {
            if (m >= g.M || n0 + c >= count) return;
            const int64_t n = first + n0 + c;
            if (bias) z += bf16_at(bias, m);
            float v;
            if constexpr (GATED) {
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
        };
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int m = m0 + (lane >> 2) + (q & 2) * 4;
                const int c = wn * 32 + j * 8 + (lane & 3) * 2 + (q & 1);
                if constexpr (GATED) {
                    finish(m + wm * 16, c, acc[0][j][q], acc[1][j][q]);
                } else {
                    finish(m + wm * 32, c, acc[0][j][q], 0.f);
                    finish(m + wm * 32 + 16, c, acc[1][j][q], 0.f);
                }
            }
    }
}

}  // namespace

cudaError_t launch_gemm_simple(const Gemm &g, cudaStream_t stream) {
    const int features = g.gated ? 64 : 128;
    const int64_t m_tiles = (static_cast<int64_t>(g.M) + features - 1) / features;
    const int64_t n_tiles = (static_cast<int64_t>(g.N) + kRowsB - 1) / kRowsB;
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
