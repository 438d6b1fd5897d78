// The grouped layout of T x K routing slots (moe_permute): a stable counting
// sort of the slots by expert, with each expert's rows padded to a tile.
//
// The slots are cut in order over CTAs, and within a CTA over warps.  A warp
// walks its run 32 slots at a time: __match_any_sync finds the lanes that
// share an expert, a lane's rank among them is the number of lower ones, and
// one lane per expert moves the warp's running count on.  Prefixes over the
// warps' and the CTAs' counts make the ranks global.  Everything is integer
// work in a fixed order, so the outputs are exact and repeatable.
//
// Two forms, both bound by latencies, not by their few megabytes:
//   - up to 8 x 16384 slots: one launch, a cluster of 1 to 8 CTAs that keeps
//     its ids and ranks in registers and exchanges counts through distributed
//     shared memory;
//   - more: three launches (counts per chunk, offsets, placement) over up to
//     304 chunks.
#include "ffn.cuh"
#include "tc.cuh"

namespace moef {
namespace {

constexpr int kPermuteThreads = 512;
constexpr int kPermuteWarps = kPermuteThreads / 32;
constexpr int kMinChunk = 2048;
constexpr int kMaxChunks = 304;

__device__ __forceinline__ int key_of(const int32_t *ids, int64_t i, int64_t n, int E) {
    if (i >= n) return E;
    const int id = __ldg(ids + i);
    return id >= 0 && id < E ? id : E;
}

constexpr int kClusterThreads = 1024;
constexpr int kClusterWarps = 32;
constexpr int kRun = 16;                        // steps of 32 slots per warp at most
constexpr int kCtaSlots = kClusterWarps * kRun * 32;
constexpr int kMaxClusterCtas = 8;

// Inclusive scan over the 1024 threads; scratch: 32 words.
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t *scratch) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) scratch[w] = v;
    __syncthreads();
    if (w == 0) {
        int32_t t = scratch[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(0xFFFFFFFFu, t, o);
            if (lane >= o) t += u;
        }
        scratch[lane] = t;
    }
    __syncthreads();
    return w ? v + scratch[w - 1] : v;
}

__device__ __forceinline__ int32_t padded_rows(int32_t count, int tile) {
    // count + tile - 1 may pass 31 bits, the padded count does not
    return static_cast<int32_t>((static_cast<int64_t>(count) + tile - 1) / tile * tile);
}

__device__ __forceinline__ int32_t load_remote_i32(uint32_t addr) {
    int32_t v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// One cluster; per_warp slots a warp (a multiple of 32, at most kRun * 32).
__global__ void __launch_bounds__(kClusterThreads)
cluster_kernel(const int32_t *ids, int n, int per_warp, int K, int E, int tile, int ctas,
               int32_t *idx_map, int32_t *row_token, int P, int32_t *offsets, int32_t *counts) {
    __shared__ int32_t scratch[32];
    extern __shared__ int32_t table[];
    int32_t *mine = table;                              // [E] slots of this CTA
    int32_t *base = table + E;                          // [E] this CTA's first row
    int32_t *pad = table + 2 * E;                       // [E] first padding row
    int32_t *next = table + 3 * E;                      // [E] the next expert's first row
    uint16_t *hist = reinterpret_cast<uint16_t *>(table + 4 * E);      // [warps][E]
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int rank = static_cast<int>(cluster_rank());

    for (int i = threadIdx.x; i < kClusterWarps * E / 2; i += kClusterThreads)
        reinterpret_cast<uint32_t *>(hist)[i] = 0u;
    allow_next_kernel();
    wait_previous_kernel();

    const int steps = per_warp / 32;
    const int i0 = (rank * kClusterWarps + w) * per_warp + lane;
    int key[kRun];
#pragma unroll
    for (int s = 0; s < kRun; ++s) {
        key[s] = E;
        if (s < steps && i0 + 32 * s < n) {
            const int id = ids[i0 + 32 * s];
            if (id >= 0 && id < E) key[s] = id;
        }
    }
    __syncthreads();

    // ranks within the warp
    uint16_t *warp_hist = hist + w * E;
    int within[kRun];
#pragma unroll
    for (int s = 0; s < kRun; ++s) {
        within[s] = 0;
        if (s < steps) {
            const unsigned same = __match_any_sync(0xFFFFFFFFu, key[s]);
            if (key[s] < E) {
                const int before = warp_hist[key[s]];
                within[s] = before + __popc(same & ((1u << lane) - 1));
                __syncwarp(same);
                if (lane == __ffs(same) - 1)
                    warp_hist[key[s]] = static_cast<uint16_t>(before + __popc(same));
            }
            __syncwarp();
        }
    }
    __syncthreads();
    // ranks within the CTA
    const int e = threadIdx.x;
    if (e < E) {
        int32_t sum = 0;
#pragma unroll 8
        for (int k = 0; k < kClusterWarps; ++k) {
            const int v = hist[k * E + e];
            hist[k * E + e] = static_cast<uint16_t>(sum);
            sum += v;
        }
        mine[e] = sum;
    }
    if (ctas > 1) cluster_sync(); else __syncthreads();
    // ranks within the cluster, offsets
    int32_t total = 0, lower = 0;
    if (e < E) {
        if (ctas > 1) {
            const uint32_t at = smem_addr(mine + e);
            int32_t v[kMaxClusterCtas];
#pragma unroll
            for (int c = 0; c < kMaxClusterCtas; ++c)
                v[c] = c < ctas ? load_remote_i32(map_rank(at, c)) : 0;
#pragma unroll
            for (int c = 0; c < kMaxClusterCtas; ++c) {
                if (c < rank) lower += v[c];
                total += v[c];
            }
        } else {
            total = mine[e];
        }
    }
    const int32_t padded = e < E ? padded_rows(total, tile) : 0;
    const int32_t end = block_scan(padded, scratch);
    if (e < E) {
        base[e] = end - padded + lower;
        pad[e] = end - padded + total;
        next[e] = end;
        if (rank == 0) {
            offsets[e] = end - padded;
            counts[e] = total;
            if (e == E - 1) offsets[E] = end;
        }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kRun; ++s) {
        const int i = i0 + 32 * s;
        if (s < steps && i < n) {
            const int k = key[s];
            const int32_t row = k < E ? base[k] + hist[w * E + k] + within[s] : -1;
            idx_map[i] = row;
            if (row >= 0) row_token[row] = i / K;
        }
    }
    // -1 on the padding rows and behind the last expert
    for (int k = rank * kClusterWarps + w; k < E; k += ctas * kClusterWarps)
        for (int r = pad[k] + lane; r < next[k]; r += 32) row_token[r] = -1;
    for (int64_t r = static_cast<int64_t>(next[E - 1]) + rank * kClusterThreads + threadIdx.x;
         r < P; r += ctas * kClusterThreads)
        row_token[r] = -1;
    if (ctas > 1) cluster_sync();       // nobody leaves while its counts may be read
}

__global__ void __launch_bounds__(kPermuteThreads)
count_kernel(const int32_t *ids, int64_t n, int64_t chunk, int E, int32_t *chunk_counts) {
    extern __shared__ int32_t hist[];
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int64_t i0 = blockIdx.x * chunk, i1 = i0 + chunk < n ? i0 + chunk : n;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += blockDim.x) {
        const int key = key_of(ids, i, n, E);
        if (key < E) atomicAdd(hist + key, 1);      // counts: the order does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        chunk_counts[static_cast<int64_t>(blockIdx.x) * E + e] = hist[e];
}

// One CTA, one thread per expert (E <= 1024 = MOEF_MAX_EXPERTS).
__global__ void __launch_bounds__(1024)
offsets_kernel(int32_t *chunk_counts, int chunks, int E, int tile, int32_t *offsets,
               int32_t *counts) {
    __shared__ int32_t scratch[32];
    const int e = threadIdx.x;
    int32_t total = 0;
    if (e < E) {
#pragma unroll 8
        for (int c = 0; c < chunks; ++c) {
            int32_t *at = chunk_counts + static_cast<int64_t>(c) * E + e;
            const int32_t v = *at;
            *at = total;
            total += v;
        }
        counts[e] = total;
    }
    const int32_t padded = padded_rows(total, tile);
    const int32_t end = block_scan(padded, scratch);
    if (e < E) {
        offsets[e] = end - padded;
        if (e == E - 1) offsets[E] = end;
    }
}

__global__ void __launch_bounds__(kPermuteThreads)
place_kernel(const int32_t *ids, int64_t n, int64_t chunk, int K, int E,
             const int32_t *chunk_base, const int32_t *offsets, const int32_t *counts,
             int32_t *idx_map, int32_t *row_token, int64_t P) {
    extern __shared__ int32_t hist[];       // [warps][E]
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kPermuteWarps * E; i += blockDim.x) hist[i] = 0;
    __syncthreads();

    const int64_t run = chunk / kPermuteWarps;      // slots per warp, a multiple of 32
    const int64_t i0 = blockIdx.x * chunk + w * run;
    // the warps' counts, then each warp's first rank within the chunk
    int32_t *mine = hist + w * E;
    for (int64_t i = i0; i < i0 + run; i += 32) {
        const int key = key_of(ids, i + lane, n, E);
        const unsigned same = __match_any_sync(0xFFFFFFFFu, key);
        if (key < E && lane == __ffs(same) - 1) mine[key] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int32_t rank = offsets[e] + chunk_base[static_cast<int64_t>(blockIdx.x) * E + e];
#pragma unroll
        for (int k = 0; k < kPermuteWarps; ++k) {
            const int32_t v = hist[k * E + e];
            hist[k * E + e] = rank;
            rank += v;
        }
    }
    __syncthreads();
    for (int64_t i = i0; i < i0 + run; i += 32) {
        const int key = key_of(ids, i + lane, n, E);
        const unsigned same = __match_any_sync(0xFFFFFFFFu, key);
        const int32_t first = key < E ? mine[key] : 0;
        const int32_t row = key < E ? first + __popc(same & ((1u << lane) - 1)) : -1;
        __syncwarp();
        if (key < E && lane == __ffs(same) - 1) mine[key] = first + __popc(same);
        __syncwarp();
        if (i + lane < n) {
            idx_map[i + lane] = row;
            if (row >= 0) row_token[row] = static_cast<int32_t>((i + lane) / K);
        }
    }

    // -1 on the padding rows and behind the last expert
    for (int e = blockIdx.x * kPermuteWarps + w; e < E; e += gridDim.x * kPermuteWarps)
        for (int64_t r = offsets[e] + counts[e] + lane; r < offsets[e + 1]; r += 32)
            row_token[r] = -1;
    for (int64_t r = offsets[E] + static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
         r < P; r += static_cast<int64_t>(gridDim.x) * blockDim.x)
        row_token[r] = -1;
}

// Slots per chunk: at least kMinChunk, at most kMaxChunks chunks, a multiple
// of 32 for each warp.
int64_t chunk_slots(int64_t n) {
    int64_t c = (n + kMaxChunks - 1) / kMaxChunks;
    if (c < kMinChunk) c = kMinChunk;
    return (c + kPermuteThreads - 1) / kPermuteThreads * kPermuteThreads;
}

}  // namespace

int permute_chunks(int64_t slots) {
    if (slots <= static_cast<int64_t>(kMaxClusterCtas) * kCtaSlots) return 0;
    const int64_t c = chunk_slots(slots);
    return static_cast<int>((slots + c - 1) / c);
}

cudaError_t launch_permute(const int32_t *ids, int T, int K, int E, int tile, int32_t *idx_map,
                           int32_t *row_token, int64_t P, int32_t *offsets, int32_t *counts,
                           int32_t *workspace, cudaStream_t stream) {
    const int64_t n = static_cast<int64_t>(T) * K;
    cudaError_t err = cudaSuccess;
    const int chunks = permute_chunks(n);
    if (chunks == 0) {
        // 64 slots a warp before the next doubling of the cluster
        int ctas = 1;
        while (ctas < kMaxClusterCtas && n > static_cast<int64_t>(ctas) * kClusterWarps * 64)
            ctas *= 2;
        const int warps = ctas * kClusterWarps;
        const int per_warp = static_cast<int>(((n + warps - 1) / warps + 31) / 32 * 32);
        const int smem = E * (4 * 4 + kClusterWarps * 2);
        if (smem > 48 * 1024) {
            err = cudaFuncSetAttribute(cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem);
            if (err != cudaSuccess) return err;
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3(kClusterThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = ctas > 1 ? 2 : 1;
        return cudaLaunchKernelEx(&cfg, cluster_kernel, ids, static_cast<int>(n), per_warp, K, E,
                                  tile, ctas, idx_map, row_token, static_cast<int>(P), offsets,
                                  counts);
    }
    const int64_t chunk = chunk_slots(n);
    const int place_smem = kPermuteWarps * E * static_cast<int>(sizeof(int32_t));
    if (place_smem > 48 * 1024)
        err = cudaFuncSetAttribute(place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   place_smem);
    if (err != cudaSuccess) return err;
    count_kernel<<<chunks, kPermuteThreads, E * sizeof(int32_t), stream>>>(ids, n, chunk, E,
                                                                            workspace);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    offsets_kernel<<<1, 1024, 0, stream>>>(workspace, chunks, E, tile, offsets, counts);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    place_kernel<<<chunks, kPermuteThreads, place_smem, stream>>>(
        ids, n, chunk, K, E, workspace, offsets, counts, idx_map, row_token, P);
    return cudaGetLastError();
}

}  // namespace moef
