// AdamW over many tensors (moe_adamw_step).
//
// Bound by HBM: a value with fp32 states and master moves 28 bytes for some forty
// operations.  A warp takes 256 values of a tensor, eight a lane (four and four, so
// that each of its accesses is one piece of memory), all its loads in flight before
// the first use; the table of tensors comes with the launch's
// parameters, so that nothing is copied or kept between calls.  256 values are also
// what an 8-bit state's scale is for, so a warp has a scale's values to itself and
// finds the largest by shuffles.  396M values: 1.56 ms with fp32 states and master
// weights (7.1 TB/s), 1.04 ms with 8-bit states (6.1 TB/s; their 75 instructions a
// value keep the SMs' issue two thirds busy).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "tc.cuh"
#include "train.cuh"
#include "vec.cuh"

namespace moef {
namespace {

constexpr int kPiece = 256;             // values a warp takes at a time
constexpr int kAdamThreads = 128;       // 8-bit states 1.04 ms, with 256 4 % more, with 512 18 %
constexpr int kEightCtas = 12;          // of an SM, with 8-bit states: 10 take 3 % more, 14 5 %
constexpr int kPerCta = kAdamThreads / 32;
constexpr float kE4m3Max = 448.f, kE4m3Least = 0.001953125f;    // 2^-9
constexpr int kFewTensors = 48, kManyTensors = 256;             // of a launch

template <int N>
struct Table {
    moef_adamw_tensor t[N];
    uint32_t end[N];                    // pieces up to each tensor's last
    int n;
};
static_assert(sizeof(Table<kManyTensors>) + sizeof(AdamWFactors) <= 32000, "launch parameters");

// Within 2^-22 of the root and the reciprocal, which the step allows.
__device__ __forceinline__ float fast_sqrt(float x) {
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Where a lane's value i is, from its first.
__device__ constexpr int place(int i) { return (i & 3) + kPiece / 2 * (i >> 2); }

// A lane's eight values of an array of `left` more (at least one), four to an access
// where `whole`.
__device__ __forceinline__ void load8(const float *p, float (&f)[8], int64_t left, bool whole) {
    if (whole) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        const float4 b = *reinterpret_cast<const float4 *>(p + kPiece / 2);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = place(i) < left ? p[place(i)] : 0.f;
    }
}
__device__ __forceinline__ void load8(const uint16_t *p, float (&f)[8], int64_t left, bool whole) {
    if (whole) {
        const uint2 a = *reinterpret_cast<const uint2 *>(p);
        const uint2 b = *reinterpret_cast<const uint2 *>(p + kPiece / 2);
        VecOps<8>::to_f32(make_uint4(a.x, a.y, b.x, b.y), f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = place(i) < left
                       ? __uint_as_float(static_cast<uint32_t>(p[place(i)]) << 16) : 0.f;
    }
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8], int64_t left, bool whole) {
    if (whole) {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(p + kPiece / 2) = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (place(i) < left) p[place(i)] = f[i];
    }
}
__device__ __forceinline__ void store8(uint16_t *p, const float (&f)[8], int64_t left,
                                       bool whole) {
    if (whole) {
        const uint4 w = VecOps<8>::from_f32(f);
        *reinterpret_cast<uint2 *>(p) = make_uint2(w.x, w.y);
        *reinterpret_cast<uint2 *>(p + kPiece / 2) = make_uint2(w.z, w.w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (place(i) < left) p[place(i)] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
    }
}

// Eight e4m3 codes as they lie in memory.
__device__ __forceinline__ uint2 load_codes(const uint8_t *p, int64_t left, bool whole) {
    uint2 c = make_uint2(0, 0);
    if (whole)
        return make_uint2(*reinterpret_cast<const uint32_t *>(p),
                          *reinterpret_cast<const uint32_t *>(p + kPiece / 2));
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (place(i) < left)
            (i < 4 ? c.x : c.y) |= static_cast<uint32_t>(p[place(i)]) << (8 * (i & 3));
    return c;
}
__device__ __forceinline__ void decode8(uint2 c, float scale, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = (i < 2 ? c.x : c.y) >> (16 * (i & 1));
        const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(pair & 0xFFFFu), __NV_E4M3));
        const float2 v = __half22float2(h);
        f[2 * i] = v.x * scale;
        f[2 * i + 1] = v.y * scale;
    }
}

// x / y and sqrt(x), rounded to nearest: an approximation and one step of Newton's
// method on its residual, which an fma gives exactly (P. Markstein, IBM J. Res. Dev.
// 34, 1990; the quotient needs y's reciprocal rounded to nearest).  Three and five
// instructions where the library's functions take about ten each, which 8-bit states
// are bound by otherwise.  The root is of 0 and of 2^-126 <= x < 2^127: below that range
// neither the approximation nor the residual is one.
__device__ __forceinline__ float rounded_quotient(float x, float y, float reciprocal) {
    const float q = x * reciprocal;
    return fmaf(fmaf(-q, y, x), reciprocal, q);
}
__device__ __forceinline__ float rounded_sqrt(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaxf(x, 1.17549435e-38f)));      // 0: 0 r
    const float s = x * r;
    return fmaf(fmaf(-s, s, x), 0.5f * r, s);
}
// Which of a lane's values these are, by the least and the largest of their patterns (the
// least of pattern - 1: 0 is not below the range).  Comparisons of each value take 5 %
// more time; zeros left to the library's root, 5 to 10 % more where there are any.
struct RootRange {
    uint32_t least = 0xFFFFFFFFu, largest = 0;
    __device__ __forceinline__ void add(float x) {
        least = min(least, __float_as_uint(x) - 1u);
        largest = max(largest, __float_as_uint(x));
    }
    __device__ __forceinline__ bool usual() const {
        return least >= 0x00800000u - 1u && largest < 0x7F000000u;
    }
};
// The largest root that is stored, 2^64 (1 - 2^-20): its code and scale give a value
// whose square is finite, so a v that passed the largest number decays again.
constexpr float kMostRoot = 0x1.ffffep63f;

// The piece's scale, and its values as codes of it.  ROOT: values above 0 keep a
// code above 0.
template <bool ROOT>
__device__ __forceinline__ void encode8(const float (&f)[8], uint8_t *p, float *scale_at, int lane,
                                        int64_t left, bool whole) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(f[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    // A code is the rounding of the rounded quotient: a product with the scale's
    // reciprocal, off by a unit in the last place, would put one value in a million
    // on the other side of a code's border, an eighth of the value away.  Scales
    // whose reciprocal is not a normal number count as 0.
    const float top = most * (1.f / kE4m3Max), scale = top > 1e-37f ? top : 0.f;
    const float reciprocal = scale > 0.f ? __frcp_rn(scale) : 0.f;
    if (lane == 0) *scale_at = scale;
    uint32_t word[2] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 v = make_float2(rounded_quotient(f[2 * i], scale, reciprocal),
                               rounded_quotient(f[2 * i + 1], scale, reciprocal));
        if constexpr (ROOT) {
            if (v.x > 0.f) v.x = fmaxf(v.x, kE4m3Least);
            if (v.y > 0.f) v.y = fmaxf(v.y, kE4m3Least);
        }
        word[i >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE,
                                                                       __NV_E4M3))
                        << (16 * (i & 1));
    }
    if (whole) {
        *reinterpret_cast<uint32_t *>(p) = word[0];
        *reinterpret_cast<uint32_t *>(p + kPiece / 2) = word[1];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (place(i) < left) p[place(i)] = static_cast<uint8_t>(word[i >> 2] >> (8 * (i & 3)));
    }
}

template <typename P, typename G, bool MASTER, bool EIGHT, int N>
__global__ void __launch_bounds__(kAdamThreads, EIGHT ? kEightCtas : 1)
adamw_kernel(const __grid_constant__ Table<N> table, const __grid_constant__ AdamWFactors f) {
    __shared__ float s_bias[2];
    const int lane = threadIdx.x & 31;
    wait_previous_kernel();
    allow_next_kernel();
    float bias1 = f.bias1, root_bias2 = f.root_bias2;
    if (f.device_step) {
        if (threadIdx.x < 2) {      // 1 - beta^step without cancellation
            const int step = max(1, *f.device_step);
            const float b = -expm1f(step * (threadIdx.x ? f.log_beta2 : f.log_beta1));
            s_bias[threadIdx.x] = threadIdx.x ? sqrtf(b) : b;
        }
        __syncthreads();
        bias1 = s_bias[0];
        root_bias2 = s_bias[1];
    }
    const float lr = f.device_lr ? *f.device_lr : f.lr;
    const float keep = 1.f - lr * f.weight_decay, step_size = lr / bias1;
    const float root = 1.f / root_bias2;
    const float grad_scale = f.grad_scale ? *f.grad_scale : 1.f;

    const uint32_t piece = blockIdx.x * kPerCta + threadIdx.x / 32;
    if (piece < table.end[table.n - 1]) {
        int at = 0;                     // the first tensor that ends behind the piece
        for (int hi = table.n - 1; at < hi;) {
            const int mid = (at + hi) >> 1;
            if (table.end[mid] > piece) hi = mid; else at = mid + 1;
        }
        const moef_adamw_tensor &t = table.t[at];
        const int64_t block = piece - (at ? table.end[at - 1] : 0);
        const int64_t i = block * kPiece + lane * 4, left = t.n - i;
        const uintptr_t bits = reinterpret_cast<uintptr_t>(t.param) |
                               reinterpret_cast<uintptr_t>(t.master) |
                               reinterpret_cast<uintptr_t>(t.grad);
        const uintptr_t states = reinterpret_cast<uintptr_t>(t.exp_avg) |
                                 reinterpret_cast<uintptr_t>(t.exp_avg_sq);
        const bool whole = left >= kPiece / 2 + 4 && bits % 16 == 0 &&
                           states % (EIGHT ? 8 : 16) == 0;
        float g[8] = {}, p[8] = {}, m[8] = {}, v[8] = {};
        if (left > 0) {
            load8(static_cast<const G *>(t.grad) + i, g, left, whole);
            if constexpr (MASTER) load8(t.master + i, p, left, whole);
            else load8(static_cast<const P *>(t.param) + i, p, left, whole);
        }
        if constexpr (EIGHT) {
            uint2 cm = make_uint2(0, 0), cv = make_uint2(0, 0);
            const float scale_m = t.exp_avg_scale[block], scale_v = t.exp_avg_sq_scale[block];
            if (left > 0) {
                cm = load_codes(static_cast<const uint8_t *>(t.exp_avg) + i, left, whole);
                cv = load_codes(static_cast<const uint8_t *>(t.exp_avg_sq) + i, left, whole);
            }
            decode8(cm, scale_m, m);
            decode8(cv, scale_v, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= v[k];
        } else if (left > 0) {
            load8(static_cast<const float *>(t.exp_avg) + i, m, left, whole);
            load8(static_cast<const float *>(t.exp_avg_sq) + i, v, left, whole);
        }
        RootRange range;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            g[k] *= grad_scale;
            m[k] = fmaf(f.rest1, g[k], __fmul_rn(f.beta1, m[k]));
            v[k] = fmaf(f.rest2, __fmul_rn(g[k], g[k]), __fmul_rn(f.beta2, v[k]));
            range.add(v[k]);
        }
        const bool usual = range.usual();
        if constexpr (EIGHT) {          // v becomes its root
            if (usual) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = rounded_sqrt(v[k]);
            } else {                    // below the normal range, near or past its end, NaN
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = sqrtf(v[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float s = EIGHT ? v[k] : fast_sqrt(v[k]);
            p[k] = fmaf(keep, p[k],
                        -(step_size * m[k]) * fast_reciprocal(fmaf(s, root, f.eps)));
        }
        if constexpr (EIGHT) {
            if (!usual) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = v[k] > kMostRoot ? kMostRoot : v[k];
            }
        }
        if (left > 0) {
            if constexpr (MASTER) store8(t.master + i, p, left, whole);
            store8(static_cast<P *>(t.param) + i, p, left, whole);
        }
        if constexpr (EIGHT) {
            encode8<false>(m, static_cast<uint8_t *>(t.exp_avg) + i, t.exp_avg_scale + block, lane,
                           left, whole);
            encode8<true>(v, static_cast<uint8_t *>(t.exp_avg_sq) + i, t.exp_avg_sq_scale + block,
                          lane, left, whole);
        } else if (left > 0) {
            store8(static_cast<float *>(t.exp_avg) + i, m, left, whole);
            store8(static_cast<float *>(t.exp_avg_sq) + i, v, left, whole);
        }
    }
}

template <typename P, typename G, bool MASTER, bool EIGHT, int N>
cudaError_t start_adamw(const moef_adamw_tensor *tensors, int n, const AdamWFactors &f,
                        cudaStream_t stream) {
    Table<N> table;
    int64_t pieces = 0;
    for (int i = 0; i < n; ++i) {
        table.t[i] = tensors[i];
        pieces += (tensors[i].n + kPiece - 1) / kPiece;
        table.end[i] = static_cast<uint32_t>(pieces);
    }
    table.n = n;
    if (pieces == 0) return cudaSuccess;
    // One piece a warp: 396M values with fp32 states and master take 1565 us, 1918
    // with four CTAs an SM that go round, 1625 with four pieces a warp, 1590 with
    // streaming hints.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((pieces + kPerCta - 1) / kPerCta));
    cfg.blockDim = dim3(kAdamThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, adamw_kernel<P, G, MASTER, EIGHT, N>, table, f);
}

template <typename P, typename G, bool MASTER, bool EIGHT>
cudaError_t start_all(const moef_adamw_tensor *tensors, int n, const AdamWFactors &f,
                      cudaStream_t stream) {
    if (n <= kFewTensors)
        return start_adamw<P, G, MASTER, EIGHT, kFewTensors>(tensors, n, f, stream);
    for (int i = 0; i < n; i += kManyTensors) {
        const cudaError_t err = start_adamw<P, G, MASTER, EIGHT, kManyTensors>(
            tensors + i, n - i < kManyTensors ? n - i : kManyTensors, f, stream);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_adamw(const moef_adamw_tensor *tensors, int n, const AdamWFactors &f,
                         int state_bits, int masters, int param_f32, int grad_f32,
                         cudaStream_t stream) {
    auto go = [&](auto *start32, auto *start8) {
        return (state_bits == 8 ? start8 : start32)(tensors, n, f, stream);
    };
    if (param_f32)
        return grad_f32 ? go(start_all<float, float, false, false>,
                             start_all<float, float, false, true>)
                        : go(start_all<float, uint16_t, false, false>,
                             start_all<float, uint16_t, false, true>);
    if (masters)
        return grad_f32 ? go(start_all<uint16_t, float, true, false>,
                             start_all<uint16_t, float, true, true>)
                        : go(start_all<uint16_t, uint16_t, true, false>,
                             start_all<uint16_t, uint16_t, true, true>);
    return grad_f32 ? go(start_all<uint16_t, float, false, false>,
                         start_all<uint16_t, float, false, true>)
                    : go(start_all<uint16_t, uint16_t, false, false>,
                         start_all<uint16_t, uint16_t, false, true>);
}

}  // namespace moef
