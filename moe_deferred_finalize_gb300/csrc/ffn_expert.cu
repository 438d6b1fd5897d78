// dz of the expert products' backward passes, over the rows of the experts alone, the
// rows of x beside it, and their bias gradients.
//
//   linear  dz = dout * act'(preact)
//   gated   dz[:, i] = dout * u * act'(g),  dz[:, n + i] = dout * act(g)
//
// dz is rounded to bf16 here, because both products take it as a bf16 operand, as the
// dense backward passes do: their outputs are then 2.3e-3 off (root mean square), of which
// their own rounding makes 1.7e-3.  A second bf16 term would double the products' work.
// dbias sums dz before that.
//
// Both are bound by HBM: dout and preact are read once, dz is written once.  The
// layout's rows are P at most, but how many the experts have only the device knows,
// and with few tokens most of P is behind the last of them (16 tokens, top-8 of
// 256, tiles of 128: 128 rows of 16384).  Each CTA counts the experts' pieces of
// eight rows itself and takes every gridDim-th of them, a row a warp.  Where there
// are fewer pieces than CTAs, a piece's columns are shared out over several (100
// tokens, two of 8 experts of 1040 x 1536: 10.2 us by 25 CTAs).
//
// dweight sums over rows, which its product copies in blocks of 64: rows of x that
// lie scattered (a row map) or cannot be copied as they are (odd sizes, misaligned
// views) are laid out once here.  Gathered by the product itself, four rows of 128
// bytes to a copy, they came at 17 bytes a clock: 32768 rows, 64 experts of 4096 x
// 7168 took 1742 us, 1259 from rows in order, which take 130 us to write.
//
// Where the layout leaves room, the rows behind an expert's last are zeros up to a
// multiple of 16 here: the product then copies its last block like the others (see
// spaced_rows).
#include "ffn.cuh"
#include "tc.cuh"
#include "train.cuh"
#include "vec.cuh"

namespace moef {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
// Vectors of a lane in flight, of each array, and CTAs: 32768 rows, 2048 gated, x of
// 7168 laid out (1.38 GB of traffic) take 225 us so (6.1 TB/s), 247 with four
// vectors, 310 with the two jobs on warps of their own.
constexpr int kLoads = 2;
constexpr int kCtasPerSm = 4;

// An expert's rows rounded up to the 16 that one step of dweight's product sums.
__device__ __forceinline__ int rounded_rows(int rows) { return (rows + 15) & ~15; }

// Rows of expert e: first, and how many, clipped to the buffer as the products clip
// them.
__device__ __forceinline__ int rows_of(const Groups &g, int e, int *first) {
    *first = g.offsets[e];
    if (*first < 0) return 0;
    const int64_t room = g.P - *first;
    return static_cast<int>(max(static_cast<int64_t>(0),
                                min(static_cast<int64_t>(g.counts[e]), room)));
}

// dz of VEC columns: out[0] (linear, or the gate's) and out[1] (the up projection's).
template <int VEC, bool GATED>
__device__ __forceinline__ void dz_of(const float (&d)[VEC], const float (&z)[VEC],
                                      const float (&u)[VEC], int act,
                                      float (&out)[GATED ? 2 : 1][VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        float a;
        const float da = act_grad(z[j], act, &a);
        if constexpr (GATED) {
            out[0][j] = d[j] * u[j] * da;
            out[1][j] = d[j] * a;
        } else {
            out[0][j] = d[j] * da;
        }
    }
}

// A row of x by a warp; without one, or outside x, zeros.
__device__ __forceinline__ void copy_row(const RowCopy &c, int64_t row, bool have, int part,
                                         int parts, int lane) {
    const int64_t token = have && c.row_token ? c.row_token[row] : row;
    have = have && token >= 0 && token < c.T;
    const uint16_t *from = c.x + (have ? token : 0) * c.K;
    uint16_t *to = c.to + row * c.pitch;
    if (c.K % 8 == 0 && reinterpret_cast<uintptr_t>(c.x) % 16 == 0) {
        const int stride = parts * 32 * 8;
        for (int i0 = (part * 32 + lane) * 8; i0 < c.K; i0 += stride * kLoads) {
            uint4 v[kLoads];
#pragma unroll
            for (int l = 0; l < kLoads; ++l) {
                v[l] = make_uint4(0, 0, 0, 0);
                if (have && i0 + stride * l < c.K)
                    v[l] = __ldg(reinterpret_cast<const uint4 *>(from + i0 + stride * l));
            }
#pragma unroll
            for (int l = 0; l < kLoads; ++l)
                if (i0 + stride * l < c.K)
                    *reinterpret_cast<uint4 *>(to + i0 + stride * l) = v[l];
        }
    } else {
        for (int i = part * 32 + lane; i < c.K; i += parts * 32) to[i] = have ? from[i] : 0;
    }
}

// dbias of one expert and a block of columns: some of a warp's lanes along the columns,
// the others along the rows (8 and 4 with 16-byte vectors: a CTA takes 64 rows at a
// time, for an expert's rows are all one CTA's: 50000 rows of one expert take 570 us,
// 64 times 512 rows 67); a warp's sums are joined by shuffles, the warps' in order.
template <int VEC>
constexpr int kColumnLanes = VEC == 8 ? 8 : 32;
template <int VEC>
constexpr int kBiasColumns = kColumnLanes<VEC> * VEC;

template <int VEC, bool GATED>
__device__ __forceinline__ void sum_bias(const uint16_t *dout, const uint16_t *preact, int act,
                                         uint16_t *dbias, const Groups &g, int n, int e, int block,
                                         float (&sums)[kWarps][GATED ? 2 : 1][kBiasColumns<VEC>]) {
    using Ops = VecOps<VEC>;
    using V = typename Ops::V;
    constexpr int kHalves = GATED ? 2 : 1, kRows = kLoads, kAcross = kColumnLanes<VEC>;
    constexpr int kStep = kWarps * (32 / kAcross);          // rows of one load of all warps
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int cols = kHalves * n, at = (lane % kAcross) * VEC, i = block * kBiasColumns<VEC> + at;
    int first;
    const int rows = rows_of(g, e, &first);
    float sum[kHalves][VEC] = {};
    for (int64_t r0 = warp * (32 / kAcross) + lane / kAcross; i < n && r0 < rows;
         r0 += kStep * kRows) {
        V d[kRows], z[kRows], u[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            if (r0 + k * kStep >= rows) break;
            const int64_t row = first + r0 + k * kStep;
            d[k] = Ops::load(dout + row * n + i);
            if (preact) z[k] = Ops::load(preact + row * cols + i);
            if constexpr (GATED) u[k] = Ops::load(preact + row * cols + n + i);
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            if (r0 + k * kStep >= rows) break;
            float df[VEC], zf[VEC] = {}, uf[VEC] = {}, out[kHalves][VEC];
            Ops::to_f32(d[k], df);
            if (preact) Ops::to_f32(z[k], zf);
            if constexpr (GATED) Ops::to_f32(u[k], uf);
            dz_of<VEC, GATED>(df, zf, uf, act, out);
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int j = 0; j < VEC; ++j) sum[h][j] += out[h][j];
        }
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
#pragma unroll
            for (int o = kAcross; o < 32; o <<= 1)
                sum[h][j] += __shfl_xor_sync(0xFFFFFFFFu, sum[h][j], o);
            if (lane < kAcross) sums[warp][h][at + j] = sum[h][j];
        }
    __syncthreads();
    for (int c = threadIdx.x; c < kHalves * kBiasColumns<VEC>; c += kThreads) {
        const int h = c / kBiasColumns<VEC>, k = c % kBiasColumns<VEC>;
        const int column = block * kBiasColumns<VEC> + k;
        if (column >= n) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += sums[w][h][k];
        dbias[static_cast<int64_t>(e) * cols + h * n + column] =
            __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
}

// One launch: the first dz_ctas CTAs make dz and lay out x, the others dbias, which
// reads the same rows at the same time (100 tokens, two of 8 experts of 1040 x 1536,
// the whole backward pass: 35.2 us with two launches, 32.9 with one).  ACT: the activation, or -1
// to take it from `act`.
template <int VEC, bool GATED, int ACT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
expert_dz_kernel(const uint16_t *dout, const uint16_t *preact, int act, uint16_t *dz,
                 int64_t pitch, uint16_t *dbias, const Groups g, int n, const RowCopy copy,
                 int dz_ctas) {
    using Ops = VecOps<VEC>;
    using V = typename Ops::V;
    struct Pieces {
        int before[MOEF_MAX_EXPERTS], first[MOEF_MAX_EXPERTS];
        int rows[MOEF_MAX_EXPERTS];     // of x, not those of zeros
        int warp[kWarps];
    };
    __shared__ union {
        Pieces pieces;
        float sums[kWarps][GATED ? 2 : 1][kBiasColumns<VEC>];
    } shared;
    int *const s_pieces = shared.pieces.before, *const s_first = shared.pieces.first;
    int *const s_rows = shared.pieces.rows, *const s_warp = shared.pieces.warp;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int cols = GATED ? 2 * n : n;
    wait_previous_kernel();
    allow_next_kernel();
    if (static_cast<int>(blockIdx.x) >= dz_ctas) {
        const unsigned across = (n - 1) / kBiasColumns<VEC> + 1, at = blockIdx.x - dz_ctas;
        sum_bias<VEC, GATED>(dout, preact, ACT < 0 ? act : ACT, dbias, g, n, at / across,
                             at % across, shared.sums);
        return;
    }
    // the pieces before each expert: a scan over four experts a thread
    constexpr int kEach = MOEF_MAX_EXPERTS / kThreads;
    int own[kEach], sum = 0, spaced = 1;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int e = threadIdx.x * kEach + i;
        own[i] = 0;
        if (e < g.E) {
            own[i] = s_rows[e] = rows_of(g, e, &s_first[e]);
            spaced &= spaced_rows(s_first[e], own[i], g.offsets[e + 1], g.P);
        }
    }
    spaced = __syncthreads_and(spaced);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (spaced) own[i] = rounded_rows(own[i]);
        own[i] = own[i] > 0 ? steps_of(own[i], kWarps) : 0;
        sum += own[i];
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31) s_warp[warp] = before;
    __syncthreads();
    before -= sum;
    int total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        s_pieces[threadIdx.x * kEach + i] = before;
        before += own[i];
    }
    __syncthreads();

    const int widest = max(n / VEC, copy.to ? copy.K / 8 : 0);      // vectors of a row
    const int parts = total > 0 ? max(1, min(dz_ctas / total, widest / 32)) : 1;
    // total * parts is at most the larger of total and the grid
    for (unsigned unit = blockIdx.x; unit < static_cast<unsigned>(total * parts);
         unit += dz_ctas) {
        const int piece = unit / parts, part = unit - piece * parts;
        int lo = 0, hi = g.E;           // s_pieces[lo] <= piece < s_pieces[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_pieces[mid] <= piece) lo = mid; else hi = mid;
        }
        const int at = (piece - s_pieces[lo]) * kWarps + warp;
        const int rows = s_rows[lo];
        if (at >= (spaced ? rounded_rows(rows) : rows)) continue;
        const int64_t row = static_cast<int64_t>(s_first[lo]) + at;
        const bool have = at < rows;
        const int stride = parts * 32 * VEC;
        if (copy.to) copy_row(copy, row, have, part, parts, lane);
        if (!have && dz) {
            const float zeros[VEC] = {};
            for (int i = (part * 32 + lane) * VEC; i < n; i += stride)
#pragma unroll
                for (int h = 0; h < (GATED ? 2 : 1); ++h)
                    *reinterpret_cast<V *>(dz + row * pitch + h * n + i) = Ops::from_f32(zeros);
            continue;
        }
        for (int i0 = (part * 32 + lane) * VEC; dz && i0 < n; i0 += stride * kLoads) {
            V d[kLoads], z[kLoads], u[kLoads];
#pragma unroll
            for (int l = 0; l < kLoads; ++l) {
                const int i = i0 + stride * l;
                if (i >= n) break;
                d[l] = Ops::load(dout + row * n + i);
                if (preact) z[l] = Ops::load(preact + row * cols + i);
                if constexpr (GATED) u[l] = Ops::load(preact + row * cols + n + i);
            }
#pragma unroll
            for (int l = 0; l < kLoads; ++l) {
                const int i = i0 + stride * l;
                if (i >= n) break;
                float df[VEC], zf[VEC] = {}, uf[VEC] = {}, out[GATED ? 2 : 1][VEC];
                Ops::to_f32(d[l], df);
                if (preact) Ops::to_f32(z[l], zf);
                if constexpr (GATED) Ops::to_f32(u[l], uf);
                dz_of<VEC, GATED>(df, zf, uf, ACT < 0 ? act : ACT, out);
                // read again by both products: an ordinary store keeps it in L2
#pragma unroll
                for (int h = 0; h < (GATED ? 2 : 1); ++h)
                    *reinterpret_cast<V *>(dz + row * pitch + h * n + i) = Ops::from_f32(out[h]);
            }
        }
    }
}

template <typename... Params, typename... Args>
cudaError_t start(void (*kernel)(Params...), dim3 grid, cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

bool vectors(const void *a, const void *b, const void *c, int n) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
                           reinterpret_cast<uintptr_t>(c);
    return n % 8 == 0 && bits % 16 == 0;
}

}  // namespace

cudaError_t launch_expert_dz(const uint16_t *dout, const uint16_t *preact, int act, int gated,
                             uint16_t *dz, int64_t pitch, uint16_t *dbias, const Groups &g, int n,
                             const RowCopy &copy, int num_sms, cudaStream_t stream) {
    const bool vec = vectors(dout, preact, dz, n);
    const int dz_ctas = dz || copy.to ? num_sms * kCtasPerSm : 0;
    const int across = vec ? kBiasColumns<8> : kBiasColumns<1>;
    const int64_t sums = dbias ? static_cast<int64_t>(g.E) * ((n - 1) / across + 1) : 0;
    const dim3 grid(static_cast<unsigned>(dz_ctas + sums));
    if (grid.x == 0) return cudaSuccess;
    auto go = [&](auto *kernel) {
        return start(kernel, grid, stream, dout, preact, act, dz, pitch, dbias, g, n, copy,
                     dz_ctas);
    };
    if (!vec)
        return gated ? go(expert_dz_kernel<1, true, -1>) : go(expert_dz_kernel<1, false, -1>);
    switch (act) {
        case MOEF_ACT_SILU:
            return gated ? go(expert_dz_kernel<8, true, MOEF_ACT_SILU>)
                         : go(expert_dz_kernel<8, false, MOEF_ACT_SILU>);
        case MOEF_ACT_GELU:
            return gated ? go(expert_dz_kernel<8, true, MOEF_ACT_GELU>)
                         : go(expert_dz_kernel<8, false, MOEF_ACT_GELU>);
        case MOEF_ACT_GELU_TANH:
            return gated ? go(expert_dz_kernel<8, true, MOEF_ACT_GELU_TANH>)
                         : go(expert_dz_kernel<8, false, MOEF_ACT_GELU_TANH>);
        case MOEF_ACT_RELU:
            return gated ? go(expert_dz_kernel<8, true, MOEF_ACT_RELU>)
                         : go(expert_dz_kernel<8, false, MOEF_ACT_RELU>);
        default:
            return gated ? go(expert_dz_kernel<8, true, MOEF_ACT_NONE>)
                         : go(expert_dz_kernel<8, false, MOEF_ACT_NONE>);
    }
}

}  // namespace moef
