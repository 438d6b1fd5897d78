// Gradients of the finalize, of the row gather and of the top-K gate.
//
// The finalize's: with r = residual_out, inv = (mean r^2 + eps)^(-1/2) and s =
// sum_h dnorm gamma r,
//
//   dr = dresidual_out + inv (dnorm gamma - r inv^2 s / H),   dm = dout + dr
//   drows[idx[t,k]] = (w scale) dm,   dweights[t,k] = scale <dm, rows[idx[t,k]]>
//
// Bound by HBM: each slot's row is read once and its gradient written once (T = 4096,
// top-8, 7168: 1.29 GB, 191 us at the copy rate), beside four to six dense rows a
// token.  dm stays in registers, in fp32, for all of a token's slots; their dot
// products are summed by shuffles, eight at a time, and then over the warps in order.
// A token is one CTA's, or, when there are few tokens, one cluster's, whose CTAs
// share its columns and join their two sums and their dot products through
// distributed shared memory (T = 16: 128 CTAs, and 8 for dgamma, 8.2 us).  CTAs go round
// the tokens and add up dgamma in shared memory, each thread its own columns, so that at
// most 1024 rows of sums are left for a kernel that adds them in order (8 us at 304 rows
// of 7168); up to 32 tokens one more cluster takes dgamma instead.  With many
// tokens the rows come through a ring (see below): 225 us at T = 4096, 0.85 of the
// copy rate.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "tc.cuh"
#include "train.cuh"
#include "vec.cuh"

namespace cg = cooperative_groups;

namespace moef {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kWarps = kMaxThreads / 32;
constexpr int kMaxSplits = 8;
constexpr int kMaxVpt = 8;
constexpr int kMaxPartials = 1024;      // rows of dgamma's sums
constexpr int kDirectTokens = 32;       // the most whose dgamma needs none
constexpr int kSlots = 8;               // of a token, in flight at a time

// How one launch is cut: `splits` CTAs (a cluster) take a token's slices of
// `slice` vectors; clusters go round the tokens.
struct Cut {
    int splits, slice, threads, vpt, nvec;
    int64_t clusters;
};

// acc[u] summed over the warp; lane 4 u has sum u.  Halving the number of values
// at each of the first steps takes 9 shuffles, 40 for eight sums by themselves.
__device__ __forceinline__ float warp_sum8(float (&acc)[8], int lane) {
#pragma unroll
    for (int half = 4, bit = 16; half >= 1; half >>= 1, bit >>= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int u = 0; u < half; ++u) {
            const float give = up ? acc[u] : acc[u + half];
            const float keep = up ? acc[u + half] : acc[u];
            acc[u] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, bit);
        }
    }
    float v = acc[0];
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
    return v;
}

// Whether dgamma is taken directly (below), without rows of sums.  One launch against
// two, in us, at H = 7168: 7.1 : 8.7 for 8 tokens, 9.4 : 10.8 for 32, 13.3 : 11.9 for 48;
// at H = 32768 19.0 : 20.6 for 32 and 34.4 : 32.5 for 48; at H = 262144 206 : 213 for 32.
// Single values, H = 32767: 39 : 41 for 16 and 81 : 48 for 24.  The sizes alone decide, as
// they do on the workspace.
bool direct_dgamma(int T, int H) { return T <= (H % 8 ? kDirectTokens / 2 : kDirectTokens); }

// dgamma of a few tokens by one cluster (or CTA) beside those that take the tokens: its
// CTAs share the tokens for their inverse RMS, which all of them get, and then the
// columns.  dnorm and r are read once more, out of L2; the launch of a kernel that sums
// rows, and the rows' workspace, are spared (T = 16, top-8, 7168: 10.2 us in two kernels).
template <int VEC, bool CLUSTER>
__device__ __forceinline__ void direct_gamma(const FinalizeBackward &p, const Cut &cut, int split) {
    using Ops = VecOps<VEC>;
    __shared__ float s_inv[kDirectTokens], s_warp[kWarps];
    const int nt = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int t = split; t < p.T; t += cut.splits) {
        float sum = 0.f;
#pragma unroll 4
        for (int v = tid; v < cut.nvec; v += nt) {
            float x[VEC];
            Ops::to_f32(Ops::load_reused(p.r + static_cast<int64_t>(t) * p.H +
                                         static_cast<int64_t>(v) * VEC), x);
#pragma unroll
            for (int q = 0; q < VEC; ++q) sum = fmaf(x[q], x[q], sum);
        }
        sum = warp_sum(sum);
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
        sum = 0.f;
        for (int w = 0; w < nt >> 5; ++w) sum += s_warp[w];
        const float inv = rsqrtf(sum / static_cast<float>(p.H) + p.eps);
        if constexpr (CLUSTER) {
            if (tid < cut.splits) *cg::this_cluster().map_shared_rank(&s_inv[t], tid) = inv;
        } else {
            if (tid == 0) s_inv[t] = inv;
        }
        __syncthreads();
    }
    if constexpr (CLUSTER) cg::this_cluster().sync();
    const int v_end = min((split + 1) * cut.slice, cut.nvec);
    for (int v = split * cut.slice + tid; v < v_end; v += nt) {
        const int64_t e = static_cast<int64_t>(v) * VEC;
        float acc[VEC] = {};
#pragma unroll 4
        for (int t = 0; t < p.T; ++t) {
            const int64_t at = static_cast<int64_t>(t) * p.H + e;
            float d[VEC], x[VEC];
            Ops::to_f32(Ops::load_reused(p.dnorm + at), d);
            Ops::to_f32(Ops::load_reused(p.r + at), x);
#pragma unroll
            for (int q = 0; q < VEC; ++q) acc[q] = fmaf(d[q] * x[q], s_inv[t], acc[q]);
        }
#pragma unroll
        for (int q = 0; q < VEC; ++q)
            p.dgamma[e + q] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[q]));
    }
}

template <int VPT, int VEC, bool NORM, bool CLUSTER>
__global__ void __launch_bounds__(kMaxThreads, VPT <= 2 ? 2 : 1)
finalize_backward_kernel(const __grid_constant__ FinalizeBackward p,
                         const __grid_constant__ Cut cut) {
    using Ops = VecOps<VEC>;
    using V = typename Ops::V;
    __shared__ int64_t s_row[2][MOEF_MAX_K];            // first value of the slot's row, -1: none
    __shared__ float s_w[2][MOEF_MAX_K];
    __shared__ float2 s_sum[2][kWarps];
    __shared__ float s_dot[2][kWarps][MOEF_MAX_K];
    __shared__ float2 s_part[2][kMaxSplits];            // the cluster's sums
    __shared__ float s_parts[2][kMaxSplits][MOEF_MAX_K];
    extern __shared__ float s_gamma[];                  // dgamma of this CTA's tokens

    const int nt = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int warps = nt >> 5, K = p.K;
    const int split = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
    const int64_t cluster = CLUSTER ? blockIdx.x / cut.splits : blockIdx.x;
    const int v_begin = split * cut.slice, v_end = min(v_begin + cut.slice, cut.nvec);
    const bool sums_gamma = NORM && p.partial;
    if (CLUSTER) cluster_arrive();
    if (sums_gamma)
        for (int i = tid; i < VPT * VEC * nt; i += nt) s_gamma[i] = 0.f;
    auto gamma_at = [&](int j, int q) -> float & {      // four values of a thread side by side
        return VEC == 8 ? s_gamma[((j * 2 + (q >> 2)) * nt + tid) * 4 + (q & 3)]
                        : s_gamma[j * nt + tid];
    };
    wait_previous_kernel();
    allow_next_kernel();
    if (CLUSTER) cluster_wait();
    if (NORM && cluster == cut.clusters) {      // one more than the tokens need
        direct_gamma<VEC, CLUSTER>(p, cut, split);
        return;
    }

    int64_t next_row = -1;
    float next_w = 0.f;
    auto fetch = [&](int64_t t) {
        if (t < p.T && tid < K) {
            const int64_t slot = t * K + tid;
            const int row = __ldg(p.idx + slot);
            next_row = row >= 0 && row < p.P ? static_cast<int64_t>(row) * p.H : -1;
            next_w = p.drows ? decode_weight(p.weights, p.wkind, slot) * p.routed_scale : 0.f;
        }
    };
    // the CTA's dot products of token t, its warps' added in order
    auto dots = [&](int par) {
        float v = 0.f;
        for (int w = 0; w < warps; ++w) v += s_dot[par][w][tid];
        return v;
    };
    fetch(cluster);
    int par = 0;
    int64_t last = -1;
    for (int64_t t = cluster; t < p.T; t += cut.clusters, par ^= 1) {
        const int64_t tok = t * p.H;
        if (tid < K) {
            s_row[par][tid] = next_row;
            s_w[par][tid] = next_w;
        }
        fetch(t + cut.clusters);
        float inv = 0.f, mean = 0.f;
        V dn[VPT] = {}, r[VPT] = {};
        if constexpr (NORM) {
            float2 sum = make_float2(0.f, 0.f);         // of r^2 and dnorm gamma r
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = v_begin + tid + j * nt;
                if (v < v_end) {
                    const int64_t e = static_cast<int64_t>(v) * VEC;
                    dn[j] = Ops::load(p.dnorm + tok + e);
                    r[j] = Ops::load(p.r + tok + e);
                }
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = v_begin + tid + j * nt;
                if (v < v_end) {
                    float d[VEC], x[VEC], g[VEC];
                    Ops::to_f32(dn[j], d);
                    Ops::to_f32(r[j], x);
                    Ops::to_f32(Ops::load_reused(p.gamma + static_cast<int64_t>(v) * VEC), g);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) {
                        sum.x = fmaf(x[q], x[q], sum.x);
                        sum.y = fmaf(d[q] * g[q], x[q], sum.y);
                    }
                }
            }
            sum.x = warp_sum(sum.x);
            sum.y = warp_sum(sum.y);
            if (lane == 0) s_sum[par][warp] = sum;
        }
        __syncthreads();
        if (!CLUSTER && last >= 0 && tid < K && p.dweights)
            p.dweights[last * K + tid] = dots(par ^ 1) * p.routed_scale;
        last = t;
        if constexpr (NORM) {
            float2 sum = make_float2(0.f, 0.f);
            for (int w = 0; w < warps; ++w) {
                sum.x += s_sum[par][w].x;
                sum.y += s_sum[par][w].y;
            }
            if constexpr (CLUSTER) {
                cg::cluster_group group = cg::this_cluster();
                if (tid < cut.splits) *group.map_shared_rank(&s_part[par][split], tid) = sum;
                group.sync();
                sum = make_float2(0.f, 0.f);
                for (int i = 0; i < cut.splits; ++i) {
                    sum.x += s_part[par][i].x;
                    sum.y += s_part[par][i].y;
                }
            }
            inv = rsqrtf(sum.x / static_cast<float>(p.H) + p.eps);
            mean = inv * inv * (sum.y / static_cast<float>(p.H));
        }
        for (int base = v_begin; base < v_end; base += nt * VPT) {
            float dm[VPT][VEC];
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = base + tid + j * nt;
#pragma unroll
                for (int q = 0; q < VEC; ++q) dm[j][q] = 0.f;
                if (v >= v_end) continue;
                const int64_t e = static_cast<int64_t>(v) * VEC;
                V d_out = {}, d_res = {};
                if (p.dres) d_res = Ops::load(p.dres + tok + e);
                if (p.dout) d_out = Ops::load(p.dout + tok + e);
                Ops::to_f32(d_res, dm[j]);
                float f[VEC];
                if constexpr (NORM) {
                    float d[VEC], x[VEC], g[VEC];
                    Ops::to_f32(dn[j], d);
                    Ops::to_f32(r[j], x);
                    Ops::to_f32(Ops::load_reused(p.gamma + e), g);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) {
                        dm[j][q] = fmaf(inv, d[q] * g[q] - x[q] * mean, dm[j][q]);
                        if (sums_gamma) gamma_at(j, q) += d[q] * x[q] * inv;
                    }
                }
                if (p.dresidual) Ops::store(p.dresidual + tok + e, Ops::from_f32(dm[j]));
                Ops::to_f32(d_out, f);
#pragma unroll
                for (int q = 0; q < VEC; ++q) dm[j][q] += f[q];
                if (p.dshared) Ops::store(p.dshared + tok + e, Ops::from_f32(dm[j]));
            }
            if (!p.drows && !p.dweights) continue;
            for (int k0 = 0; k0 < K; k0 += kSlots) {
                float acc[kSlots] = {};
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int v = base + tid + j * nt;
                    if (v >= v_end) continue;
                    const int64_t e = static_cast<int64_t>(v) * VEC;
                    V x[kSlots] = {};
                    if (p.dweights) {
#pragma unroll
                        for (int u = 0; u < kSlots; ++u)
                            if (k0 + u < K && s_row[par][k0 + u] >= 0)
                                x[u] = Ops::load_row(p.rows + s_row[par][k0 + u] + e);
                    }
#pragma unroll
                    for (int u = 0; u < kSlots; ++u) {
                        if (k0 + u >= K || s_row[par][k0 + u] < 0) continue;
                        float f[VEC];
                        Ops::to_f32(x[u], f);
#pragma unroll
                        for (int q = 0; q < VEC; ++q) acc[u] = fmaf(f[q], dm[j][q], acc[u]);
                        if (p.drows) {
                            const float w = s_w[par][k0 + u];
#pragma unroll
                            for (int q = 0; q < VEC; ++q) f[q] = w * dm[j][q];
                            Ops::store(p.drows + s_row[par][k0 + u] + e, Ops::from_f32(f));
                        }
                    }
                }
                const float v = warp_sum8(acc, lane);
                const int k = k0 + (lane >> 2);
                if ((lane & 3) == 0 && k < K) {
                    float *at = &s_dot[par][warp][k];
                    *at = base == v_begin ? v : *at + v;
                }
            }
        }
        if constexpr (CLUSTER) {
            __syncthreads();
            cg::cluster_group group = cg::this_cluster();
            if (tid < K) *group.map_shared_rank(&s_parts[par][split][tid], 0) = dots(par);
            group.sync();
            if (split == 0 && tid < K && p.dweights) {
                float v = 0.f;
                for (int i = 0; i < cut.splits; ++i) v += s_parts[par][i][tid];
                p.dweights[t * K + tid] = v * p.routed_scale;
            }
        }
    }
    if (!CLUSTER && last >= 0) {
        __syncthreads();
        if (tid < K && p.dweights) p.dweights[last * K + tid] = dots(par ^ 1) * p.routed_scale;
    }
    if (sums_gamma) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = v_begin + tid + j * nt;
            if (v < v_end)
#pragma unroll
                for (int q = 0; q < VEC; ++q)
                    p.partial[cluster * p.H + static_cast<int64_t>(v) * VEC + q] = gamma_at(j, q);
        }
    }
}

// 16 bytes of global memory into this thread's shared memory, asynchronously, and the
// groups that such copies are waited for by.
__device__ __forceinline__ void copy_async(uint32_t to, const uint16_t *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void commit_group() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void wait_groups() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The same for many tokens and rows of 16-byte pieces, 8192 values at most (a row's pieces
// are all in one CTA's registers; longer ones, without the norm, stay with the plain form:
// T = 4096, top-8, 16384 takes 352 us, 337 at the copy rate): one CTA a token, two CTAs an SM,
// and what a token reads comes through a ring of NS rows in shared memory, one item
// (a row of dnorm, r, dresidual_out or dout, then the slots' rows) behind the other,
// across tokens: NS - 1 items are in flight while the CTA sums, waits at its barrier or
// writes.  Every thread copies, waits for and reads its own pieces alone, so the ring
// needs no barrier.  The plain form above reads nothing while it sums a token's r: T =
// 4096, top-8, 7168 with RMSNorm took 254 us (5.1 TB/s).
template <int VPT, int NS, bool NORM>
__global__ void __launch_bounds__(kMaxThreads, 2)
finalize_backward_ring_kernel(const __grid_constant__ FinalizeBackward p,
                              const __grid_constant__ Cut cut) {
    using Ops = VecOps<8>;
    constexpr int kAhead = NS - 1;
    __shared__ int64_t s_row[3][MOEF_MAX_K];    // of this token and the next: the third is being filled
    __shared__ float s_w[3][MOEF_MAX_K];
    __shared__ float2 s_sum[2][kWarps];
    __shared__ float s_dot[2][kWarps][MOEF_MAX_K];
    extern __shared__ __align__(16) float s_ring[];     // NS rows, then dgamma's sums

    const int nt = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int warps = nt >> 5, K = p.K, step = static_cast<int>(cut.clusters);
    const bool sums_gamma = NORM && p.dgamma;
    float4 *s_gamma = reinterpret_cast<float4 *>(s_ring + NS * VPT * nt * 4);
    const uint32_t ring = smem_addr(s_ring) + tid * 16;
    const uint32_t slot_bytes = VPT * nt * 16;
    if (sums_gamma)
#pragma unroll
        for (int j = 0; j < 2 * VPT; ++j) s_gamma[j * nt + tid] = make_float4(0.f, 0.f, 0.f, 0.f);
    wait_previous_kernel();
    allow_next_kernel();

    const int dense = (NORM ? 2 : 0) + (p.dres ? 1 : 0) + (p.dout ? 1 : 0);
    const int items = dense + K;
    int64_t next_row = -1;
    float next_w = 0.f;
    auto fetch = [&](int64_t t) {
        next_row = -1;
        if (t < p.T && tid < K) {
            const int64_t slot = t * K + tid;
            const int row = __ldg(p.idx + slot);
            next_row = row >= 0 && row < p.P ? static_cast<int64_t>(row) * p.H : -1;
            next_w = p.drows ? decode_weight(p.weights, p.wkind, slot) * p.routed_scale : 0.f;
        }
    };
    auto put = [&](int buf) {
        if (tid < K) {
            s_row[buf][tid] = next_row;
            s_w[buf][tid] = next_w;
        }
    };
    // Copies item i of token t (row numbers in s_row[buf]) into ring slot `to`; nothing
    // where there is none, but always a group.
    auto issue = [&](int64_t t, int i, int buf, int to) {
        if (t < p.T) {
            const uint16_t *from = nullptr;
            if (i < dense) {
                if (NORM && i < 2) from = i == 0 ? p.dnorm : p.r;
                else from = p.dres && i == (NORM ? 2 : 0) ? p.dres : p.dout;
                from += t * p.H;
            } else if (p.dweights && s_row[buf][i - dense] >= 0) {
                from = p.rows + s_row[buf][i - dense];
            }
            if (from) {
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int v = tid + j * nt;
                    if (v < cut.nvec)
                        copy_async(ring + to * slot_bytes + j * nt * 16, from + v * 8);
                }
            }
        }
        commit_group();
    };
    int64_t t = blockIdx.x;
    int buf = 0, slot = 0, par = 0;
    auto after = [](int b) { return b == 2 ? 0 : b + 1; };
    // item i of token t: waits for it, reads it, and sends for the one kAhead further
    auto take = [&](int i, uint4 (&x)[VPT]) {
        wait_groups<kAhead - 1>();
#pragma unroll
        for (int j = 0; j < VPT; ++j) x[j] = shared_load16(ring + slot * slot_bytes + j * nt * 16);
        const int before = slot == 0 ? NS - 1 : slot - 1;       // read in the last step
        if (i + kAhead < items) issue(t, i + kAhead, buf, before);
        else issue(t + step, i + kAhead - items, after(buf), before);
        slot = slot + 1 == NS ? 0 : slot + 1;
    };
    auto dots = [&](int which) {
        float v = 0.f;
        for (int w = 0; w < warps; ++w) v += s_dot[which][w][tid];
        return v;
    };
    fetch(t);
    put(0);
    fetch(t + step);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) issue(t, i, 0, i);         // items >= kAhead + 2

    int64_t last = -1;
    for (; t < p.T; t += step, buf = after(buf), par ^= 1) {
        const int64_t tok = t * p.H;
        put(after(buf));
        fetch(t + 2 * static_cast<int64_t>(step));
        float inv = 0.f, mean = 0.f;
        uint4 dn[VPT], r[VPT];
        if constexpr (NORM) {
            take(0, dn);
            take(1, r);
            float2 sum = make_float2(0.f, 0.f);         // of r^2 and dnorm gamma r
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = tid + j * nt;
                if (v < cut.nvec) {
                    float d[8], x[8], g[8];
                    Ops::to_f32(dn[j], d);
                    Ops::to_f32(r[j], x);
                    Ops::to_f32(Ops::load_reused(p.gamma + v * 8), g);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        sum.x = fmaf(x[q], x[q], sum.x);
                        sum.y = fmaf(d[q] * g[q], x[q], sum.y);
                    }
                }
            }
            sum.x = warp_sum(sum.x);
            sum.y = warp_sum(sum.y);
            if (lane == 0) s_sum[par][warp] = sum;
        }
        __syncthreads();        // and the next token's rows may be sent for
        if (last >= 0 && tid < K && p.dweights)
            p.dweights[last * K + tid] = dots(par ^ 1) * p.routed_scale;
        last = t;
        if constexpr (NORM) {
            float2 sum = make_float2(0.f, 0.f);
            for (int w = 0; w < warps; ++w) {
                sum.x += s_sum[par][w].x;
                sum.y += s_sum[par][w].y;
            }
            inv = rsqrtf(sum.x / static_cast<float>(p.H) + p.eps);
            mean = inv * inv * (sum.y / static_cast<float>(p.H));
        }
        // both gradients are here before either output is written, which may be them
        float dm[VPT][8] = {};
        uint4 d_out[VPT] = {};
        int i = NORM ? 2 : 0;
        if (p.dres) {
            take(i++, d_out);
#pragma unroll
            for (int j = 0; j < VPT; ++j) Ops::to_f32(d_out[j], dm[j]);
        }
        if (p.dout) take(i++, d_out);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * nt;
            if (v >= cut.nvec) continue;
            if constexpr (NORM) {
                float d[8], x[8], g[8];
                Ops::to_f32(dn[j], d);
                Ops::to_f32(r[j], x);
                Ops::to_f32(Ops::load_reused(p.gamma + v * 8), g);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    dm[j][q] = fmaf(inv, d[q] * g[q] - x[q] * mean, dm[j][q]);
                if (sums_gamma) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float4 &s = s_gamma[(2 * j + h) * nt + tid];
                        float4 a = s;
                        a.x += d[4 * h] * x[4 * h] * inv;
                        a.y += d[4 * h + 1] * x[4 * h + 1] * inv;
                        a.z += d[4 * h + 2] * x[4 * h + 2] * inv;
                        a.w += d[4 * h + 3] * x[4 * h + 3] * inv;
                        s = a;
                    }
                }
            }
            if (p.dresidual) Ops::store(p.dresidual + tok + v * 8, Ops::from_f32(dm[j]));
        }
        if (p.dout) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                float f[8];
                Ops::to_f32(d_out[j], f);
#pragma unroll
                for (int q = 0; q < 8; ++q) dm[j][q] += f[q];
            }
        }
        if (p.dshared) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = tid + j * nt;
                if (v < cut.nvec) Ops::store(p.dshared + tok + v * 8, Ops::from_f32(dm[j]));
            }
        }
        for (int k0 = 0; k0 < K; k0 += kSlots) {
            float acc[kSlots] = {};
#pragma unroll
            for (int u = 0; u < kSlots; ++u) {
                const int k = k0 + u;
                if (k >= K) break;
                uint4 x[VPT];
                take(i++, x);
                const int64_t row = s_row[buf][k];
                if (row < 0) continue;
                const float w = s_w[buf][k];
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int v = tid + j * nt;
                    if (v >= cut.nvec) continue;
                    float f[8];
                    if (p.dweights) {
                        Ops::to_f32(x[j], f);
#pragma unroll
                        for (int q = 0; q < 8; ++q) acc[u] = fmaf(f[q], dm[j][q], acc[u]);
                    }
                    if (p.drows) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) f[q] = w * dm[j][q];
                        Ops::store(p.drows + row + v * 8, Ops::from_f32(f));
                    }
                }
            }
            const float v = warp_sum8(acc, lane);
            const int k = k0 + (lane >> 2);
            if ((lane & 3) == 0 && k < K) s_dot[par][warp][k] = v;
        }
    }
    if (last >= 0) {
        __syncthreads();
        if (tid < K && p.dweights) p.dweights[last * K + tid] = dots(par ^ 1) * p.routed_scale;
    }
    wait_groups<0>();
    if (sums_gamma) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * nt;
            if (v < cut.nvec)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float4 *>(p.partial + static_cast<int64_t>(blockIdx.x) * p.H +
                                                v * 8 + 4 * h) = s_gamma[(2 * j + h) * nt + tid];
        }
    }
}

// dgamma = the column sums of partial [rows, H]: 32 columns a CTA, its warps every
// sixteenth row each, added in order.
constexpr int kSumWarps = 16;

__global__ void __launch_bounds__(32 * kSumWarps)
gamma_sum_kernel(const float *partial, uint16_t *dgamma, int rows, int H) {
    __shared__ float sums[kSumWarps][32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
    wait_previous_kernel();
    allow_next_kernel();
    float sum = 0.f;
    if (c < H) {
#pragma unroll 16
        for (int i = warp; i < rows; i += kSumWarps) sum += partial[static_cast<int64_t>(i) * H + c];
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < H) {
#pragma unroll
        for (int w = 1; w < kSumWarps; ++w) sum += sums[w][lane];
        dgamma[c] = __bfloat16_as_ushort(__float2bfloat16_rn(sum));
    }
}

template <typename... Params, typename... Args>
cudaError_t start(void (*kernel)(Params...), int64_t grid, int threads, size_t smem, int cluster,
                  cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

template <int VPT, int VEC, bool NORM, bool CLUSTER>
cudaError_t start_backward(const FinalizeBackward &p, const Cut &cut, cudaStream_t stream) {
    auto *kernel = finalize_backward_kernel<VPT, VEC, NORM, CLUSTER>;
    const size_t smem = NORM && p.partial ? sizeof(float) * VPT * VEC * cut.threads : 0;
    constexpr int kMost = sizeof(float) * VPT * VEC * kMaxThreads;
    if (NORM && kMost > 32 * 1024) {    // the same for every call: threads may race to set it
        const cudaError_t err = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (err != cudaSuccess) return err;
    }
    const int64_t clusters = cut.clusters + (p.dgamma && !p.partial);
    return start(kernel, clusters * cut.splits, cut.threads, smem, cut.splits, stream, p, cut);
}

template <int VPT, int VEC>
cudaError_t start_backward(const FinalizeBackward &p, const Cut &cut, cudaStream_t stream) {
    // more than two vectors a thread: rows with RMSNorm over the largest cluster alone
    if constexpr (VPT > 2)
        return start_backward<VPT, VEC, true, true>(p, cut, stream);
    else if (p.dnorm)
        return cut.splits > 1 ? start_backward<VPT, VEC, true, true>(p, cut, stream)
                              : start_backward<VPT, VEC, true, false>(p, cut, stream);
    else
        return cut.splits > 1 ? start_backward<VPT, VEC, false, true>(p, cut, stream)
                              : start_backward<VPT, VEC, false, false>(p, cut, stream);
}

template <int VEC>
cudaError_t start_backward(const FinalizeBackward &p, const Cut &cut, cudaStream_t stream) {
    switch (cut.vpt) {
        case 1: return start_backward<1, VEC>(p, cut, stream);
        case 2: return start_backward<2, VEC>(p, cut, stream);
        case 4: return start_backward<4, VEC>(p, cut, stream);
        default: return start_backward<8, VEC>(p, cut, stream);
    }
}

// The ring's form, when a token has enough items for it, the CTA's threads have a whole
// row between them (without RMSNorm rows may be longer: the plain form goes over them in
// steps) and its pieces are few enough for two CTAs an SM; false (nothing launched)
// otherwise.
constexpr int kRingBytes = 102 * 1024;

template <int VPT, int NS>
bool start_ring(const FinalizeBackward &p, Cut cut, cudaStream_t stream, cudaError_t *err) {
    const int items = (p.dnorm ? 2 : 0) + (p.dres ? 1 : 0) + (p.dout ? 1 : 0) + p.K;
    const int pieces = VPT * cut.threads;
    const size_t smem = static_cast<size_t>(pieces) * 16 * (NS + (p.dnorm && p.dgamma ? 2 : 0));
    if (items < NS + 1 || pieces < cut.nvec || smem > kRingBytes) return false;
    auto *kernel = p.dnorm ? finalize_backward_ring_kernel<VPT, NS, true>
                           : finalize_backward_ring_kernel<VPT, NS, false>;
    *err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (*err == cudaSuccess)
        *err = start(kernel, cut.clusters, cut.threads, smem, 1, stream, p, cut);
    return true;
}

bool start_ring(const FinalizeBackward &p, const Cut &cut, cudaStream_t stream,
                cudaError_t *err) {
    if (cut.vpt == 1)
        return start_ring<1, 6>(p, cut, stream, err) || start_ring<1, 4>(p, cut, stream, err);
    return cut.vpt == 2 && (start_ring<2, 5>(p, cut, stream, err) ||
                            start_ring<2, 4>(p, cut, stream, err));
}

bool vector_rows(int H, std::initializer_list<const void *> pointers) {
    uintptr_t bits = 0;
    for (const void *q : pointers) bits |= reinterpret_cast<uintptr_t>(q);
    return H % 8 == 0 && bits % 16 == 0;
}

// ------------------------------------------------------------- row gather

constexpr int kUnpermuteThreads = 128;

// A thread sums one vector of a token: its slots' rows, eight loads in flight, and
// what is added.  Bound by HBM at T = 16384 (2.58 GB in 360 us, 7.2 TB/s); T = 256
// takes 7.9 us, 5.1 of them its bytes.
template <int VEC>
__global__ void __launch_bounds__(kUnpermuteThreads)
unpermute_kernel(const __grid_constant__ Unpermute p, int nvec, int slices) {
    using Ops = VecOps<VEC>;
    using V = typename Ops::V;
    __shared__ int64_t s_row[MOEF_MAX_K];
    const int64_t t = blockIdx.x / slices;
    const int v = (blockIdx.x - t * slices) * kUnpermuteThreads + threadIdx.x;
    wait_previous_kernel();
    allow_next_kernel();
    if (threadIdx.x < p.K) {
        const int row = __ldg(p.idx + t * p.K + threadIdx.x);
        s_row[threadIdx.x] = row >= 0 && row < p.P ? static_cast<int64_t>(row) * p.H : -1;
    }
    const int64_t e = static_cast<int64_t>(v) * VEC, at = t * p.H + e;
    V add[2] = {};
    if (v < nvec) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (p.add[i]) add[i] = Ops::load(p.add[i] + at);
    }
    __syncthreads();
    if (v >= nvec) return;
    float acc[VEC] = {}, f[VEC];
    for (int k0 = 0; k0 < p.K; k0 += kSlots) {
        V x[kSlots] = {};
#pragma unroll
        for (int u = 0; u < kSlots; ++u)
            if (k0 + u < p.K && s_row[k0 + u] >= 0) x[u] = Ops::load_row(p.rows + s_row[k0 + u] + e);
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
            Ops::to_f32(x[u], f);
#pragma unroll
            for (int q = 0; q < VEC; ++q) acc[q] += f[q];
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        Ops::to_f32(add[i], f);
#pragma unroll
        for (int q = 0; q < VEC; ++q) acc[q] += f[q];
    }
    Ops::store(p.out + at, Ops::from_f32(acc));
}

// ------------------------------------------------------------------- gate

constexpr int kGateThreads = 128;

// A warp takes a token: the row is written as zeros, and then lane k puts slot k's
// value into it (the warp's barrier orders the two).  Bound by the writes at large T
// (comparing every column with every id took 9.4 us at T = 16384 and 256 experts, as
// many instructions as the bytes have time for eight times over).
template <typename T, int VEC>
__global__ void __launch_bounds__(kGateThreads)
gate_backward_kernel(const __grid_constant__ GateBackward p) {
    const int lane = threadIdx.x & 31, K = p.K;
    wait_previous_kernel();
    allow_next_kernel();
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kGateThreads / 32);
    for (int64_t t = blockIdx.x * static_cast<int64_t>(kGateThreads / 32) + threadIdx.x / 32;
         t < p.T; t += warps) {
        int id = -1;
        float w = 0.f, dw = 0.f;
        if (lane < K) {
            id = p.ids[t * K + lane];
            if (id < 0 || id >= p.E) id = -1;
            if (id >= 0) {
                w = p.weights[t * K + lane];
                dw = p.dweights[t * K + lane];
            }
        }
        float d = w * (dw - warp_sum(w * dw));
        if (p.kind == MOEF_GATE_SIGMOID && id >= 0)
            d *= 1.f / (1.f + expf(p.logits[t * p.E + id]));
        T *row = static_cast<T *>(p.dlogits) + t * p.E;
        for (int c = lane * VEC; c < p.E; c += 32 * VEC) {
            if constexpr (VEC == 1) row[c] = 0;
            else *reinterpret_cast<uint4 *>(row + c) = make_uint4(0, 0, 0, 0);
        }
        // a token that names an expert twice: its first slot has the sum, in slot order
        const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
        const bool first = id >= 0 && (same & ((1u << lane) - 1)) == 0;
        if (__any_sync(0xFFFFFFFFu, id >= 0 && !first)) {
            float sum = 0.f;
            for (int k = 0; k < K; ++k) {
                const float dk = __shfl_sync(0xFFFFFFFFu, d, k);
                if (same >> k & 1) sum += dk;
            }
            d = sum;
        }
        __syncwarp();
        if (first) {
            if constexpr (sizeof(T) == 4) row[id] = d;
            else row[id] = __bfloat16_as_ushort(__float2bfloat16_rn(d));
        }
    }
}

}  // namespace

int finalize_backward_partials(int T, int H) {
    return direct_dgamma(T, H) ? 0 : T < kMaxPartials ? T : kMaxPartials;
}

bool finalize_backward_fits(int64_t nvec) {
    return nvec <= static_cast<int64_t>(kMaxThreads) * kMaxVpt * kMaxSplits;
}

cudaError_t launch_finalize_backward(const FinalizeBackward &p, int num_sms,
                                     cudaStream_t stream) {
    const bool vec = vector_rows(p.H, {p.rows, p.r, p.gamma, p.dout, p.dres, p.dnorm, p.drows,
                                       p.dshared, p.dresidual});
    Cut cut;
    cut.nvec = vec ? p.H / 8 : p.H;
    cut.splits = 1;
    while (cut.splits < kMaxSplits &&
           (2 * static_cast<int64_t>(p.T) * cut.splits <= 4 * num_sms && cut.nvec >= 64 * cut.splits ||
            p.dnorm && cut.nvec > static_cast<int64_t>(kMaxThreads) * 2 * cut.splits))
        cut.splits *= 2;
    cut.slice = (cut.nvec - 1) / cut.splits + 1;
    cut.splits = (cut.nvec - 1) / cut.slice + 1;        // none is empty
    cut.vpt = 1;
    while (cut.vpt < (p.dnorm ? kMaxVpt : 2) && cut.slice > kMaxThreads * cut.vpt) cut.vpt *= 2;
    const int need = (cut.slice - 1) / cut.vpt + 1;
    cut.threads = need < kMaxThreads ? (need + 31) / 32 * 32 : kMaxThreads;
    int64_t clusters = static_cast<int64_t>(num_sms) * (2048 / cut.threads) / 2 / cut.splits;
    if (clusters < 1) clusters = 1;
    if (clusters > kMaxPartials) clusters = kMaxPartials;
    cut.clusters = clusters < p.T ? clusters : p.T;
    cudaError_t err = cudaSuccess;
    if (!vec || cut.splits > 1 || (p.dgamma && !p.partial) || !start_ring(p, cut, stream, &err))
        err = vec ? start_backward<8>(p, cut, stream) : start_backward<1>(p, cut, stream);
    if (err == cudaSuccess && p.partial)
        err = start(gamma_sum_kernel, (p.H - 1) / 32 + 1, 32 * kSumWarps, 0, 1, stream, p.partial, p.dgamma,
                    static_cast<int>(cut.clusters), p.H);
    return err;
}

int64_t unpermute_ctas(int T, int H) {
    return static_cast<int64_t>(T) * ((H - 1) / kUnpermuteThreads + 1);
}

cudaError_t launch_unpermute(const Unpermute &p, cudaStream_t stream) {
    const bool vec = vector_rows(p.H, {p.rows, p.add[0], p.add[1], p.out});
    const int nvec = vec ? p.H / 8 : p.H;
    const int slices = (nvec - 1) / kUnpermuteThreads + 1;
    const int64_t grid = static_cast<int64_t>(p.T) * slices;
    return vec ? start(unpermute_kernel<8>, grid, kUnpermuteThreads, 0, 1, stream, p, nvec, slices)
               : start(unpermute_kernel<1>, grid, kUnpermuteThreads, 0, 1, stream, p, nvec, slices);
}

cudaError_t launch_gate_backward(const GateBackward &p, int num_sms, cudaStream_t stream) {
    const int64_t need = (static_cast<int64_t>(p.T) + kGateThreads / 32 - 1) / (kGateThreads / 32);
    const int64_t most = static_cast<int64_t>(num_sms) * 16;
    const int64_t grid = need < most ? need : most;
    const bool vec = reinterpret_cast<uintptr_t>(p.dlogits) % 16 == 0 && p.E % (p.f32 ? 4 : 8) == 0;
    if (p.f32)
        return start(vec ? gate_backward_kernel<float, 4> : gate_backward_kernel<float, 1>, grid,
                     kGateThreads, 0, 1, stream, p);
    return start(vec ? gate_backward_kernel<uint16_t, 8> : gate_backward_kernel<uint16_t, 1>, grid,
                 kGateThreads, 0, 1, stream, p);
}

}  // namespace moef
