// The forward products of moe_ffn.h for a handful of rows (decode): bound by
// reading the weights once, so nothing stands between HBM and the registers.
//
// A CTA owns 16 rows of A (8 gate and the 8 up rows in the gated form) and
// splits k over its warps, 64 values a step.  The products use mma.m16n8k16
// with the lanes' loads as they come: the sum over k does not care which k a
// fragment slot holds, as long as A and B agree, so a lane's 16-byte load of
// row g (8 consecutive k) is taken as the k slots of two MMAs, and the same
// 16 bytes of token g feed the B side.  No shared memory, no transposition
// before the warps' partial sums meet at the end.  Each warp has four steps (8
// KB of weights) in flight, 16 warps an SM.
//
// Against the tensor-core kernel with k split over a cluster it saves the
// pipeline set-up, two cluster barriers and the remote reads.
#include "ffn.cuh"
#include "tc.cuh"
#include "vec.cuh"

namespace moef {
namespace {

constexpr int kStepK = 64;

// Plain loads: the previous kernel on the stream, whose tail this one may share
// the SM with, can have written any operand.
__device__ __forceinline__ uint4 load_once(const uint16_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// The same, or zeros.
__device__ __forceinline__ uint4 load_if(const uint16_t *p, bool ok) {
    uint4 v;
    asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %5, 0;\n"
                 "mov.u32 %0, 0;\nmov.u32 %1, 0;\nmov.u32 %2, 0;\nmov.u32 %3, 0;\n"
                 "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
                 : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
                 : "l"(p), "r"(static_cast<uint32_t>(ok)));
    return v;
}

__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 k values of rows g (lo) and g + 8 (hi) against 8 of the token.
__device__ __forceinline__ void mma_16bytes(float (&c)[4], const uint4 &lo, const uint4 &hi,
                                            const uint4 &x) {
    mma16(c, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
    mma16(c, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
}

__device__ __forceinline__ float bf16_or_zero(const uint16_t *p, int64_t i) {
    return p ? __uint_as_float(static_cast<uint32_t>(p[i]) << 16) : 0.f;
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// features: output features of this CTA, at most 16 (8 gated); fewer leave MMA
// rows empty and spread a small matrix over more SMs.
template <bool GATED, int W>
__global__ void __launch_bounds__(32 * W, 16 / W)
decode_kernel(const Gemm g, const int features) {
    __shared__ float part[W][16][kDecodeRows + 1];
    constexpr int kDepth = 4;                   // steps in flight per warp
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int m0 = blockIdx.x * features;
    const int row = lane >> 2, k8 = (lane & 3) * 8;

    // Rows and tokens that are not there read an existing one: their sums are
    // not used.
    const int lo_row = row < features && m0 + row < g.M ? m0 + row : m0;
    const int hi_row = GATED ? g.M + lo_row
                       : row + 8 < features && m0 + row + 8 < g.M ? m0 + row + 8 : m0;
    const uint16_t *a_lo = g.a + static_cast<int64_t>(lo_row) * g.K + k8;
    const uint16_t *a_hi = g.a + static_cast<int64_t>(hi_row) * g.K + k8;
    const uint16_t *x = g.b + static_cast<int64_t>(row < g.N ? row : 0) * g.K + k8;

    wait_previous_kernel();
    allow_next_kernel();

    float acc[4] = {};
    const int full = g.K / kStepK, steps = (g.K + kStepK - 1) / kStepK;
    int s0 = warp;
    for (; s0 + W * (kDepth - 1) < full; s0 += W * kDepth) {
        uint4 lo[kDepth][2], hi[kDepth][2], xv[kDepth][2];
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = (s0 + d * W) * kStepK + 32 * j;
                lo[d][j] = load_once(a_lo + k);
                hi[d][j] = load_once(a_hi + k);
                xv[d][j] = load_once(x + k);
            }
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
#pragma unroll
            for (int j = 0; j < 2; ++j) mma_16bytes(acc, lo[d][j], hi[d][j], xv[d][j]);
    }
    if (s0 < steps) {       // fewer than kDepth steps, the last one maybe partial
        uint4 lo[kDepth][2], hi[kDepth][2], xv[kDepth][2];
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = (s0 + d * W) * kStepK + 32 * j;
                const bool in = k + k8 < g.K;
                lo[d][j] = load_if(a_lo + k, in);
                hi[d][j] = load_if(a_hi + k, in);
                xv[d][j] = load_if(x + k, in);
            }
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
#pragma unroll
            for (int j = 0; j < 2; ++j) mma_16bytes(acc, lo[d][j], hi[d][j], xv[d][j]);
    }
    const int c = (lane & 3) * 2;
    part[warp][row][c] = acc[0];
    part[warp][row][c + 1] = acc[1];
    part[warp][row + 8][c] = acc[2];
    part[warp][row + 8][c + 1] = acc[3];
    __syncthreads();

    // the warps' sums in warp order, features along the threads
    for (int i = threadIdx.x; i < features * g.N; i += 32 * W) {
        const int r = i % features, n = i / features, m = m0 + r;
        if (m >= g.M) continue;
        float z = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            z += part[w][r][n];
            if constexpr (GATED) u += part[w][r + 8][n];
        }
        z += bf16_or_zero(g.bias, m);
        const int64_t at = static_cast<int64_t>(n) * g.M + m;
        float v;
        if constexpr (GATED) {
            u += bf16_or_zero(g.bias, g.M + m);
            if (g.preact) {
                g.preact[at + static_cast<int64_t>(n) * g.M] = bf16_bits(z);
                g.preact[at + static_cast<int64_t>(n + 1) * g.M] = bf16_bits(u);
            }
            v = act_value(z, g.act) * u;
        } else {
            if (g.preact) g.preact[at] = bf16_bits(z);
            v = act_value(z, g.act);
            if (g.residual)
                v += __uint_as_float(static_cast<uint32_t>(g.residual[at]) << 16);
        }
        if (g.out_f32) static_cast<float *>(g.out)[at] = v;
        else static_cast<uint16_t *>(g.out)[at] = bf16_bits(v);
    }
}

template <int W>
cudaError_t start(const Gemm &g, int ctas, int features, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(32 * W);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return g.gated ? cudaLaunchKernelEx(&cfg, decode_kernel<true, W>, g, features)
                   : cudaLaunchKernelEx(&cfg, decode_kernel<false, W>, g, features);
}

// Features per CTA: whole MMA rows when they give every SM a CTA, else down to
// a quarter of them: 256 router rows run on 64 CTAs instead of 16.
int features_per_cta(const Gemm &g, int num_sms) {
    int features = g.gated ? 8 : 16;
    const int least = features / 4;
    while (features > least && (g.M + features - 1) / features < num_sms) features /= 2;
    return features;
}

// Whether this kernel or the tensor-core one is faster, from sweeps (us): this
// one starts in 1.5 and reads 6.9 MB/us, but a round of its CTAs takes at least
// 1.8, more than a short k needs; the other one starts in 3.8 and reads 6.7
// MB/us.  1 x 65536 x 512: 25 here, 13.7 there; 1 x 4096 x 7168: 11.3 and 12.7;
// 1 x 65536 x 7168: 131-134 and 138, 8 rows of it 135-139 and 138.  From 9 rows
// on, a second fragment of tokens made this one slower than the other everywhere
// but at a router's size (16 x 4096 x 7168: 13.9 and 12.8; 16 x 256 x 7168: 6.1
// and 6.4).
bool pays(const Gemm &g, int ctas, int num_sms) {
    const double mb = 2e-6 * g.M * (g.gated ? 2.0 : 1.0) * g.K;
    const int at_once = (ctas <= num_sms ? 1 : ctas <= 2 * num_sms ? 2 : 4) * num_sms;
    const double latency = 1.8 * ((ctas + at_once - 1) / at_once), read = mb / 6.9;
    return 1.5 + (read > latency ? read : latency) < 3.8 + mb / 6.7;
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

bool launch_gemm_decode(const Gemm &g, int num_sms, cudaStream_t stream, cudaError_t *err) {
    if (g.E || g.a_mn || g.b_mn || g.N > kDecodeRows || g.K % 8 || g.b_pitch != g.K ||
        !aligned16(g.a) || !aligned16(g.b))
        return false;
    const int features = features_per_cta(g, num_sms);
    const int ctas = (g.M + features - 1) / features;
    if (!pays(g, ctas, num_sms)) return false;
    // The SMs hold 16 warps of this kernel (128 registers): one CTA of 16, two
    // of 8 or four of 4, whichever gets most CTAs running at once (65536 rows
    // of 7168: 136 us in CTAs of 8 warps, 131 of 4; 8192 of 1024: 5.5 and 4.8).
    *err = ctas <= num_sms       ? start<16>(g, ctas, features, stream)
           : ctas <= 2 * num_sms ? start<8>(g, ctas, features, stream)
                                 : start<4>(g, ctas, features, stream);
    return true;
}

}  // namespace moef
