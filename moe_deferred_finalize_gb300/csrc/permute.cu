// The grouped layout of T x K routing slots (moe_permute): a stable counting
// sort of the slots by expert, with each expert's rows padded to a tile.
//
// The slots are cut into chunks in order.  Pass 1 counts each chunk's slots
// per expert; pass 2 (one CTA) turns the counts into each chunk's first rank
// within each expert, and the padded totals into offsets; pass 3 ranks the
// slots within their chunk and writes the maps.  Everything is integer work
// in a fixed order, so the outputs are exact and repeatable.
//
// Within a chunk each warp walks a contiguous run of slots, 32 at a time:
// __match_any_sync finds the lanes that share an expert, a lane's rank among
// them is the number of lower ones, and one lane per expert moves the warp's
// running count on.  A prefix over the warps' counts makes the ranks those of
// the chunk.
#include "ffn.cuh"

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
    __shared__ int32_t warp_total[32];
    const int e = threadIdx.x, lane = e & 31, w = e >> 5;
    int32_t total = 0;
    if (e < E) {
        for (int c = 0; c < chunks; ++c) {
            int32_t *at = chunk_counts + static_cast<int64_t>(c) * E + e;
            const int32_t v = *at;
            *at = total;
            total += v;
        }
        counts[e] = total;
    }
    const int32_t padded =      // total + tile - 1 may pass 31 bits, the padded count does not
        static_cast<int32_t>((static_cast<int64_t>(total) + tile - 1) / tile * tile);
    int32_t sum = padded;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) warp_total[w] = sum;
    __syncthreads();
    int32_t before = 0;
    for (int k = 0; k < w; ++k) before += warp_total[k];
    if (e < E) {
        offsets[e] = before + sum - padded;
        if (e == E - 1) offsets[E] = before + sum;
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
    for (int e = blockIdx.x; e < E; e += gridDim.x)
        for (int64_t r = offsets[e] + counts[e] + threadIdx.x; r < offsets[e + 1];
             r += blockDim.x)
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
    const int64_t c = chunk_slots(slots);
    return slots ? static_cast<int>((slots + c - 1) / c) : 1;
}

cudaError_t launch_permute(const int32_t *ids, int T, int K, int E, int tile, int32_t *idx_map,
                           int32_t *row_token, int64_t P, int32_t *offsets, int32_t *counts,
                           int32_t *workspace, cudaStream_t stream) {
    const int64_t n = static_cast<int64_t>(T) * K;
    const int64_t chunk = chunk_slots(n);
    const int chunks = permute_chunks(n);
    const int place_smem = kPermuteWarps * E * static_cast<int>(sizeof(int32_t));
    cudaError_t err = cudaSuccess;
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
