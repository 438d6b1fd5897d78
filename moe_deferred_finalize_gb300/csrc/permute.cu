// The grouped layout of T x K routing slots (moe_permute): a stable counting
// sort of the slots by expert, with each expert's rows padded to a tile.
//
// The slots are cut in order over CTAs, and within a CTA over warps.  A warp
// walks its run 32 slots at a time: one ballot per bit of the expert id finds
// the lanes that share an expert (__match_any_sync took 500 clocks a step), a
// lane's rank among them is the number of lower ones, and one lane per expert
// moves the warp's running count on.  Prefixes over the warps' and the CTAs'
// counts make the ranks global.  Everything is integer work in a fixed order,
// so the outputs are exact and repeatable.
//
// Two forms, both bound by latencies and by scattered 4-byte stores, not by
// their few megabytes:
//   - up to 16384 slots: one launch, a cluster of up to 8 CTAs that keeps its
//     ids and ranks in registers and exchanges counts through distributed
//     shared memory;
//   - more: two launches over up to 304 chunks, one for the chunks' counts and
//     one that places; every CTA of the second sums the counts it needs.
#include "ffn.cuh"
#include "tc.cuh"

namespace moef {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRun = 8;                         // steps of 32 slots per warp in the cluster form
constexpr int kCtaSlots = kWarps * kRun * 32;
constexpr int kMaxCtas = 8;
constexpr int kMinChunk = 512, kMidChunk = 2048;
constexpr int kMaxChunks = 304;
constexpr int kPer = MOEF_MAX_EXPERTS / kThreads;       // experts per thread at most

// Tables in shared memory, each [E].
struct Tables {
    int32_t *total;     // the expert's slots
    int32_t *base;      // this CTA's first row (first: its slots before this CTA)
    int32_t *pad;       // first padding row
    int32_t *next;      // the next expert's first row
};

__device__ __forceinline__ Tables tables(int32_t *smem, int E) {
    return {smem, smem + E, smem + 2 * E, smem + 3 * E};
}

__device__ __forceinline__ int key_of(int id, int E) { return id >= 0 && id < E ? id : E; }

// The lanes of the warp that hold the same key (0 .. E).
__device__ __forceinline__ unsigned same_key(int key, int E) {
    unsigned same = 0xFFFFFFFFu;
#pragma unroll
    for (int b = 0; b < 11; ++b) {
        if (E >> b == 0) break;
        const unsigned with = __ballot_sync(0xFFFFFFFFu, key & (1 << b));
        same &= key & (1 << b) ? with : ~with;
    }
    return same;
}

// t.total and t.base (slots before this CTA) -> t.base, t.pad, t.next, and the
// outputs when `write`.
__device__ __forceinline__ void place_experts(const Tables &t, int E, int tile, bool write,
                                              int32_t *offsets, int32_t *counts) {
    __shared__ int32_t warp_sum[kWarps];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int per = (E + kThreads - 1) / kThreads, e0 = threadIdx.x * per;
    int32_t padded[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        padded[j] = 0;
        if (j < per && e0 + j < E)      // total + tile - 1 may pass 31 bits, this does not
            padded[j] = static_cast<int32_t>(
                (static_cast<int64_t>(t.total[e0 + j]) + tile - 1) / tile * tile);
        sum += padded[j];
    }
    int32_t scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) warp_sum[w] = scan;
    __syncthreads();
    int32_t first = scan - sum;
    for (int k = 0; k < w; ++k) first += warp_sum[k];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = e0 + j;
        if (j < per && e < E) {
            t.base[e] += first;
            t.pad[e] = first + t.total[e];
            t.next[e] = first + padded[j];
            if (write) {
                offsets[e] = first;
                counts[e] = t.total[e];
                if (e == E - 1) offsets[E] = first + padded[j];
            }
            first += padded[j];
        }
    }
    __syncthreads();
}

// A lane's first padding row: the layout may end at row 2^31 - 1, which the sum passes.
__device__ __forceinline__ constexpr int64_t padding_row(int32_t pad, int lane) {
    return static_cast<int64_t>(pad) + lane;
}
static_assert(padding_row(INT32_MAX, 31) == int64_t{INT32_MAX} + 31, "64-bit rows");

// -1 on the padding rows and behind the last expert, shared by `ctas` CTAs.
__device__ __forceinline__ void fill_padding(const Tables &t, int E, int32_t *row_token,
                                             int64_t P, int cta, int ctas) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int e = cta * kWarps + w; e < E; e += ctas * kWarps)
        for (int64_t r = padding_row(t.pad[e], lane); r < t.next[e]; r += 32)
            row_token[r] = -1;
    for (int64_t r = t.next[E - 1] + static_cast<int64_t>(cta) * kThreads + threadIdx.x; r < P;
         r += static_cast<int64_t>(ctas) * kThreads)
        row_token[r] = -1;
}

__device__ __forceinline__ int32_t load_remote_i32(uint32_t addr) {
    int32_t v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// One cluster of `ctas` CTAs; `steps` steps of 32 slots a warp.
__global__ void __launch_bounds__(kThreads)
cluster_kernel(const int32_t *ids, int n, int steps, int K, int E, int tile, int ctas,
               int32_t *idx_map, int32_t *row_token, int P, int32_t *offsets, int32_t *counts) {
    extern __shared__ int32_t smem[];
    const Tables t = tables(smem, E);
    int32_t *mine = smem + 4 * E;                               // [E] slots of this CTA
    uint16_t *hist = reinterpret_cast<uint16_t *>(smem + 5 * E);        // [warps][E]
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int rank = static_cast<int>(cluster_rank());

    for (int i = threadIdx.x; i < kWarps * E / 2; i += kThreads)
        reinterpret_cast<uint32_t *>(hist)[i] = 0u;
    wait_previous_kernel();
    allow_next_kernel();

    const int i0 = (rank * kWarps + w) * steps * 32 + lane;
    int key[kRun], within[kRun];
#pragma unroll
    for (int s = 0; s < kRun; ++s)
        key[s] = s < steps && i0 + 32 * s < n ? ids[i0 + 32 * s] : E;
    __syncthreads();
    // ranks within the warp
    uint16_t *warp_hist = hist + w * E;
#pragma unroll
    for (int s = 0; s < kRun; ++s) {
        key[s] = key_of(key[s], E);
        if (s >= steps) break;
        const unsigned same = same_key(key[s], E);
        const int before = key[s] < E ? warp_hist[key[s]] : 0;
        within[s] = before + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (key[s] < E && lane == __ffs(same) - 1)
            warp_hist[key[s]] = static_cast<uint16_t>(before + __popc(same));
        __syncwarp();
    }
    __syncthreads();
    // ranks within the CTA
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int32_t sum = 0;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const int v = hist[k * E + e];
            hist[k * E + e] = static_cast<uint16_t>(sum);
            sum += v;
        }
        mine[e] = sum;
    }
    if (ctas > 1) cluster_sync(); else __syncthreads();
    // ranks within the cluster
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int32_t v[kMaxCtas], lower = 0, total = 0;
        const uint32_t at = smem_addr(mine + e);
#pragma unroll
        for (int c = 0; c < kMaxCtas; ++c)
            v[c] = c >= ctas ? 0 : ctas > 1 ? load_remote_i32(map_rank(at, c)) : mine[e];
#pragma unroll
        for (int c = 0; c < kMaxCtas; ++c) {
            if (c < rank) lower += v[c];
            total += v[c];
        }
        t.total[e] = total;
        t.base[e] = lower;
    }
    __syncthreads();
    place_experts(t, E, tile, rank == 0, offsets, counts);
#pragma unroll
    for (int s = 0; s < kRun; ++s) {
        const int i = i0 + 32 * s, k = key[s];
        if (s < steps && i < n) {
            const int32_t row = k < E ? t.base[k] + hist[w * E + k] + within[s] : -1;
            idx_map[i] = row;
            if (row >= 0) row_token[row] = i / K;
        }
    }
    fill_padding(t, E, row_token, P, rank, ctas);
    if (ctas > 1) cluster_sync();       // nobody leaves while its counts may be read
}

// Slots per expert of each chunk.
__global__ void __launch_bounds__(kThreads)
count_kernel(const int32_t *ids, int64_t n, int64_t chunk, int E, int32_t *chunk_counts) {
    extern __shared__ int32_t smem[];
    for (int e = threadIdx.x; e < E; e += kThreads) smem[e] = 0;
    wait_previous_kernel();
    allow_next_kernel();
    __syncthreads();
    const int64_t i0 = blockIdx.x * chunk, i1 = i0 + chunk < n ? i0 + chunk : n;
#pragma unroll 8
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
        const int key = key_of(ids[i], E);
        if (key < E) atomicAdd(smem + key, 1);      // counts: the order does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads)
        chunk_counts[static_cast<int64_t>(blockIdx.x) * E + e] = smem[e];
}

__global__ void __launch_bounds__(kThreads)
place_kernel(const int32_t *ids, int64_t n, int64_t chunk, int K, int E, int tile,
             const int32_t *chunk_counts, int32_t *idx_map, int32_t *row_token, int64_t P,
             int32_t *offsets, int32_t *counts) {
    extern __shared__ int32_t smem[];
    const Tables t = tables(smem, E);
    int32_t *hist = smem + 4 * E;                   // [warps][E]
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kWarps * E; i += kThreads) hist[i] = 0;
    wait_previous_kernel();
    allow_next_kernel();
    __syncthreads();

    // the warps' counts
    const int64_t run = chunk / kWarps;             // slots per warp, a multiple of 32
    const int64_t i0 = blockIdx.x * chunk + w * run + lane;
    int32_t *mine = hist + w * E;
#pragma unroll 8
    for (int64_t i = i0; i < i0 + run; i += 32) {
        const int key = i < n ? key_of(ids[i], E) : E;
        if (key < E) atomicAdd(mine + key, 1);      // counts: the order does not matter
    }
    // the chunks' counts
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int32_t lower = 0, total = 0;
#pragma unroll 32
        for (int c = 0; c < static_cast<int>(gridDim.x); ++c) {
            const int32_t v = chunk_counts[static_cast<int64_t>(c) * E + e];
            if (c < static_cast<int>(blockIdx.x)) lower += v;
            total += v;
        }
        t.total[e] = total;
        t.base[e] = lower;
    }
    __syncthreads();
    place_experts(t, E, tile, blockIdx.x == 0, offsets, counts);
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int32_t row = t.base[e];
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const int32_t v = hist[k * E + e];
            hist[k * E + e] = row;
            row += v;
        }
    }
    __syncthreads();
#pragma unroll 4
    for (int64_t i = i0; i < i0 + run; i += 32) {
        const int key = i < n ? key_of(ids[i], E) : E;
        const unsigned same = same_key(key, E);
        const int32_t first = key < E ? mine[key] : 0;
        __syncwarp();
        if (key < E && lane == __ffs(same) - 1) mine[key] = first + __popc(same);
        __syncwarp();
        if (i < n) {
            const int32_t row = key < E ? first + __popc(same & ((1u << lane) - 1)) : -1;
            idx_map[i] = row;
            if (row >= 0) row_token[row] = static_cast<int32_t>(i / K);
        }
    }
    fill_padding(t, E, row_token, P, blockIdx.x, gridDim.x);
}

// Slots per chunk, a multiple of 32 for each warp.  A chunk's ranking takes its
// slots' time, summing the chunks' counts theirs: 64 chunks of 512 to 2048
// slots (32768 slots: 8.2 us, with 16 chunks of 2048 10.7; 131072 slots: 12.4,
// with 128 chunks of 1024 21.7), then up to kMaxChunks, then longer ones.
int64_t chunk_slots(int64_t n) {
    int64_t c = (n + 63) / 64;
    if (c < kMinChunk) c = kMinChunk;
    if (c > kMidChunk) c = kMidChunk;
    if (n > c * kMaxChunks) c = (n + kMaxChunks - 1) / kMaxChunks;
    return (c + kThreads - 1) / kThreads * kThreads;
}

template <typename... Params, typename... Args>
cudaError_t start(void (*kernel)(Params...), int ctas, int cluster, int smem,
                  cudaStream_t stream, Args... args) {
    if (smem > 47 * 1024) {         // static shared memory counts towards the 48 KB too
        const cudaError_t err = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err != cudaSuccess) return err;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
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

}  // namespace

int permute_chunks(int64_t slots) {
    if (slots <= static_cast<int64_t>(kMaxCtas) * kCtaSlots) return 0;
    const int64_t c = chunk_slots(slots);
    return static_cast<int>((slots + c - 1) / c);
}

cudaError_t launch_permute(const int32_t *ids, int T, int K, int E, int tile, int32_t *idx_map,
                           int32_t *row_token, int64_t P, int32_t *offsets, int32_t *counts,
                           int32_t *workspace, cudaStream_t stream) {
    const int64_t n = static_cast<int64_t>(T) * K;
    const int chunks = permute_chunks(n);
    if (chunks == 0) {
        // One step a warp until the cluster is full; the padding rows share
        // its CTAs too, so a few slots with many of those take them as well.
        const int64_t work = n > P / 16 ? n : P / 16;
        int ctas = 1;
        while (ctas < kMaxCtas && work > static_cast<int64_t>(ctas) * kThreads) ctas *= 2;
        const int steps = static_cast<int>((n + ctas * kThreads - 1) / (ctas * kThreads));
        return start(cluster_kernel, ctas, ctas, E * (5 * 4 + kWarps * 2), stream, ids, n, steps,
                     K, E, tile, ctas, idx_map, row_token, P, offsets, counts);
    }
    const int64_t chunk = chunk_slots(n);
    const cudaError_t err = start(count_kernel, chunks, 1, E * 4, stream, ids, n, chunk, E,
                                  workspace);
    if (err != cudaSuccess) return err;
    return start(place_kernel, chunks, 1, E * 4 * (4 + kWarps), stream, ids, n, chunk, K, E, tile,
                 workspace, idx_map, row_token, P, offsets, counts);
}

}  // namespace moef
