// The products of moe_ffn.h on the tensor cores (tcgen05, TMA).
//
// out[n, m] = epilogue(sum_k A[m, k] B[n, k]): the MMA's M side carries the
// output features, its N side the tokens.  That way one token or 256 use the
// same instruction (N is any multiple of 16), ragged expert groups waste at
// most 31 columns, and every product of a layer reads its operands as they
// lie, k-contiguous or m-contiguous (the descriptor's transpose bits).
//
// A CTA is sixteen warps.  One issues the TMA copies of 64-deep k blocks of A
// into a ring of shared-memory stages (128-byte swizzle), another those of B;
// one warp for both needed 430 clocks a block, near the 512 that the MMAs of
// the widest tile take.  Gathered rows are copied four to an instruction, so B
// then has six warps (64 experts of 4096 x 1536, 32768 rows: 1681 us with one
// warp, 659 with four, 589 with six).  One lane of a further warp issues the MMAs
// into TMEM, and eight warps finish tiles, twelve when the gathering ones are free
// (4096 x 4864 x 64, bound by its epilogue: 16.5 us with eight, 14.5 with twelve;
// with a residual 29.8 and 25.1).  The accumulator is double buffered (2 x 256
// TMEM columns), so a tile's epilogue runs under the next tile's products.
//
// Gated form: the A tile interleaves gate and up rows, which one tensor map of
// the weights does in the copy: eight of each in turn ([E][I / 8][2][8][H]), so
// that a gate and its up value come into one thread's fragments.  Where the
// number of features is not a multiple of 8, or an output is not 16-byte
// aligned, the rows alternate one by one ([E][I][2][H]), and two shuffles a pair
// of columns bring the values together.
//
// The two gradients of a layer are independent and often fill the last round of
// tiles badly; they run as one launch over both products' tiles when that is
// priced lower (746 x 2512 x 4968: 43 us apart, 36.5 together).
//
// Two launch forms:
//   CG = 2  pairs of CTAs share tiles of 256 (m) x up to 256 (n): each CTA
//           loads half of A and half of B, one instruction drives both SMs'
//           tensor cores.  Persistent, one pair per two SMs.
//   CG = 1  128 x up to 256 tiles: few tokens give few tiles, which spread over
//           all SMs.
// k can also be split over a cluster of `split` CTAs or pairs: each finishes
// its share of the tile's columns, the others send it their sums of those
// into its shared memory, and it adds them in rank order (equal calls give
// equal bits).  Expert groups choose the split on the device, where the number
// of tiles is known: a cluster's units share one tile's k, or take tiles alone.
#include <stddef.h>

#include "ffn.cuh"
#include "host.cuh"
#include "tc.cuh"
#include "vec.cuh"

namespace moef {
namespace {

constexpr int kCopyWarp = 10;                   // copies B; warp 0 copies A
constexpr int kBiasWarp = kCopyWarp + 1;        // sums bias gradients
constexpr int kGatherWarps = 6;                 // copy B from kCopyWarp on when rows are gathered
constexpr int kGatherLanes = (32 + kGatherWarps - 1) / kGatherWarps;   // of each; 4 rows a lane
constexpr int kTcThreads = 32 * (kCopyWarp + kGatherWarps);
constexpr int kBlockK = 64;                     // k values per stage: one 128-byte swizzle row
constexpr int kATile = 128 * kBlockK * 2;       // bytes of A per CTA and stage
constexpr int kMaxBn = 256;
constexpr int kMaxStages = 16;
constexpr int kHeader = 13 * 1024;              // barriers, tables
constexpr int kStash = 1024;                    // bytes of each epilogue warp
constexpr int kStashes = 12 * kStash;           // over the tables when there are no groups
constexpr int kSmemBytes = 227 * 1024;
constexpr int kStageArea = kSmemBytes - kHeader - 1024;     // after rounding up to 1024
constexpr int kBand = 8;                        // feature tiles per band (see tile_at)
constexpr long long kWaitLimit = 4000000000;     // clocks (two seconds) until a wait gives up
constexpr long long kBlockLimit = 4096;          // more for each k block that it waits for

// How one launch is cut up (see choose_cut).
struct TcPlan {
    int log_split;      // 2^log_split parts of k; groups: at most, chosen on the device
    int received;       // bytes of the other parts' sums (not groups)
    int bn;             // columns per tile; groups: at most, they follow from the counts
    int m_tiles, n_tiles;
    int gather;         // B rows are fetched by row_token
    int box_rows;       // rows of one B copy (k-contiguous B)
    int wide_rows;      // of one copy through the third map, while that many are left (0: none)
    int vectors;        // rows of the output are whole, aligned 16-byte pieces
};

// One launch: a product, or two that share the SMs (the gradients of a layer):
// tiles below tiles0 are the first one's.
template <int N>
struct Work {
    CUtensorMap map[N][3];      // A, B, B in wide copies
    Gemm g[N];
    TcPlan p[N];
    int tiles0;
    BiasSum bias;
};

struct Header {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
    uint32_t tmem;
    int gave_up;
    int bn;
    int tiles;
    int log_split;
    // expert groups: column tiles before each, first row, rows
    int prefix[MOEF_MAX_EXPERTS + 1], first[MOEF_MAX_EXPERTS], count[MOEF_MAX_EXPERTS];
};
static_assert(sizeof(Header) <= kHeader && offsetof(Header, prefix) <= kHeader - kStashes,
              "header region");

__device__ unsigned int lost_waits;

// Waits for a barrier's phase; false when the wait gave up (here or in
// another warp of the CTA), upon which every role leaves its loops.  Only time
// in which the warp ran counts: a gap between two looks at the clock (the
// process lost its time slice) counts as kGap at most.  A whole tile's wait has
// its k blocks added: dweight of 2^31 - 1 rows takes 2 million of 460 ns a CTA.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *gave_up,
                                     int blocks = 0) {
    if (bar_try(bar, parity)) return true;
    constexpr long long kGap = 1 << 20;
    long long last = clock64(), spent = 0;
    for (int i = 1; !bar_try(bar, parity); ++i) {
        if (i % 64) continue;
        if (*gave_up) return false;
        const long long now = clock64();
        spent += min(now - last, kGap);
        last = now;
        if (spent > kWaitLimit + blocks * kBlockLimit) {
            *gave_up = 1;
            atomicAdd(&lost_waits, 1u);
            return false;
        }
    }
    return true;
}

// Shared-memory matrix descriptors, 128-byte swizzle.  k-contiguous: 8-row
// groups 1024 bytes apart.  m-contiguous: blocks of 64 m, each 64 k rows of
// 128 bytes; 8-k groups 1024 bytes apart, m blocks 8192.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, int mn) {
    const uint32_t lo = ((addr & 0x3FFFF) >> 4) | ((mn ? 8192u >> 4 : 1u) << 16);
    const uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

struct Tile {
    int64_t row0;       // first output row
    int count;          // valid columns (output rows)
    int bn;             // columns computed
    int m0;             // first feature
    int e;              // expert
};

template <int CG, bool GATED>
__device__ __forceinline__ Tile tile_at(const Gemm &g, const TcPlan &p, const Header *h, int t) {
    constexpr int kFeatures = (GATED ? 64 : 128) * CG;
    Tile r;
    r.e = 0;
    int m, n;
    if (g.E) {
        int lo = 0, hi = g.E;           // prefix[lo] * m_tiles <= t < prefix[hi] * m_tiles
        const int column = t / p.m_tiles;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (h->prefix[mid] <= column) lo = mid; else hi = mid;
        }
        r.e = lo;
        const int nt = h->prefix[lo + 1] - h->prefix[lo];
        const int local = t - h->prefix[lo] * p.m_tiles;
        const int count = h->count[lo];
        int columns = count - 1;
        m = local;
        n = 0;
        if (nt > 1) {       // the quotients cost 4 % of 57 tokens on 128 experts of 5112 x 88
            m = local / nt;
            n = local - m * nt;
            columns /= nt;
        }
        r.bn = (columns + 16 * CG) / (16 * CG) * (16 * CG);
        r.row0 = static_cast<int64_t>(h->first[lo]) + n * r.bn;
        r.count = min(r.bn, count - n * r.bn);
    } else {
        // bands of kBand feature tiles, columns outside: the tiles in flight form
        // a block, so both operands are shared through L2
        const unsigned per_band = kBand * p.n_tiles, band = static_cast<unsigned>(t) / per_band;
        const unsigned in_band = t - band * per_band;
        const unsigned wide = min(kBand, p.m_tiles - static_cast<int>(band) * kBand);
        n = wide == kBand ? in_band / kBand : in_band / wide;
        m = band * kBand + in_band - n * wide;
        r.bn = p.bn;
        r.row0 = static_cast<int64_t>(n) * r.bn;
        r.count = static_cast<int>(min(static_cast<int64_t>(r.bn), g.N - r.row0));
    }
    r.m0 = m * kFeatures;
    return r;
}

// ------------------------------------------------------------- epilogue

__device__ __forceinline__ float bf16_value(const uint16_t *p, int64_t i) {
    return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}

__device__ __forceinline__ void store_pair(uint16_t *p, int64_t i, float a, float b, bool both,
                                           bool vec) {
    const uint32_t v = pack_bf16x2(a, b);
    if (vec) {
        *reinterpret_cast<uint32_t *>(p + i) = v;
    } else {
        p[i] = static_cast<uint16_t>(v);
        if (both) p[i + 1] = static_cast<uint16_t>(v >> 16);
    }
}

// Finishes the adjacent features m, m + 1 of output rows; per-thread constants
// of a tile.  vec: pairs are whole and aligned, one access each.
template <bool GATED>
struct Finish {
    const Gemm &g;
    int m;
    bool any, both, vec;
    float bias[GATED ? 4 : 2];

    // e: the expert whose bias is loaded; negative: none
    __device__ __forceinline__ Finish(const Gemm &gemm, int feature, int e) : g(gemm), m(feature) {
        any = m < g.M;
        both = m + 1 < g.M;
        const uintptr_t out = reinterpret_cast<uintptr_t>(g.out);
        const uintptr_t rest = reinterpret_cast<uintptr_t>(g.residual) |
                               reinterpret_cast<uintptr_t>(g.preact);
        vec = (g.M & 1) == 0 && (rest & 3) == 0 && (out & (g.out_f32 ? 7 : 3)) == 0;
        const uint16_t *b = g.bias + static_cast<int64_t>(e) * (GATED ? 2 : 1) * g.M;
        const bool have = e >= 0 && g.bias != nullptr;
        bias[0] = have && any ? bf16_value(b, m) : 0.f;
        bias[1] = have && both ? bf16_value(b, m + 1) : 0.f;
        if constexpr (GATED) {
            bias[2] = have && any ? bf16_value(b, g.M + m) : 0.f;
            bias[3] = have && both ? bf16_value(b, g.M + m + 1) : 0.f;
        }
    }

    __device__ __forceinline__ uint32_t residual(int64_t n) const {
        const uint16_t *p = g.residual + n * g.M + m;
        if (vec) return *reinterpret_cast<const uint32_t *>(p);
        return static_cast<uint32_t>(p[0]) | (both ? static_cast<uint32_t>(p[1]) << 16 : 0u);
    }

    // Linear: z0, z1 of row n (bias added), res its residual pair.
    __device__ __forceinline__ void linear(int64_t n, float z0, float z1, uint32_t res) const {
        const int64_t i = n * g.M + m;
        if (g.preact) store_pair(g.preact, i, z0, z1, both, vec);
        if (g.act != MOEF_ACT_NONE) {
            z0 = act_value(z0, g.act);
            z1 = act_value(z1, g.act);
        }
        if (g.residual) {
            z0 += bf16_lo(res);
            z1 += bf16_hi(res);
        }
        if (!g.out_f32) {
            store_pair(static_cast<uint16_t *>(g.out), i, z0, z1, both, vec);
        } else {
            float *o = static_cast<float *>(g.out) + i;
            if (vec) {
                *reinterpret_cast<float2 *>(o) = make_float2(z0, z1);
            } else {
                o[0] = z0;
                if (both) o[1] = z1;
            }
        }
    }

    __device__ __forceinline__ void gated(int64_t n, float g0, float g1, float u0,
                                          float u1) const {
        if (g.preact) {
            store_pair(g.preact, n * 2 * g.M + m, g0, g1, both, vec);
            store_pair(g.preact, n * 2 * g.M + g.M + m, u0, u1, both, vec);
        }
        store_pair(static_cast<uint16_t *>(g.out), n * g.M + m, act_value(g0, g.act) * u0,
                   act_value(g1, g.act) * u1, both, vec);
    }
};

// act over an array, the choice outside the loop so that its elements overlap.
template <int N>
__device__ __forceinline__ void act_all(float (&z)[N], int act) {
#define MOEF_ACT_LOOP(A)                                        \
    case A:                                                     \
        _Pragma("unroll") for (int i = 0; i < N; ++i) z[i] = act_value(z[i], A); \
        break;
    switch (act) {
        MOEF_ACT_LOOP(MOEF_ACT_SILU)
        MOEF_ACT_LOOP(MOEF_ACT_GELU)
        MOEF_ACT_LOOP(MOEF_ACT_GELU_TANH)
        MOEF_ACT_LOOP(MOEF_ACT_RELU)
        default: break;
    }
#undef MOEF_ACT_LOOP
}

__device__ __forceinline__ void store2(uint16_t *p, float a, float b) {
    *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(a, b);
}

// A pair by itself: for views whose pairs cannot be one access (odd feature
// counts, 2-byte aligned outputs).
template <bool GATED>
__device__ __noinline__ void finish_scalar(const Gemm &g, int m, int64_t n, float a, float b,
                                           float c, float d) {
    const Finish<GATED> f(g, m, -1);
    if constexpr (GATED) f.gated(n, a, b, c, d);
    else f.linear(n, a, b, g.residual ? f.residual(n) : 0u);
}

constexpr int kChunk = 16;      // columns a warp finishes at a time

// A warp's part of one tile: its 32 lanes (rows of A), every second or third chunk
// (one for each of the `sides` warps of these lanes) of the columns [begin, end).
// Made before the accumulator is waited for, so that the bias and the first
// chunk's residual are there by then.
template <bool GATED>
struct TilePart {
    const Finish<GATED> f;
    const Tile t;
    int lane, quarter, first, stride, own, begin, end;
    uint32_t next[GATED ? 1 : kChunk / 2];      // residual pairs of the next chunk

    __device__ __forceinline__ TilePart(const Gemm &g, const Tile &tile, int m_cta, int warp_quarter,
                                        int side, int sides, int warp_lane, int from, int to)
        : f(g, m_cta + (GATED ? warp_quarter * 16 + (warp_lane >> 2) * 2
                              : warp_quarter * 32 + (warp_lane & ~1)), tile.e),
          t(tile), lane(warp_lane), quarter(warp_quarter), first(from + kChunk * side),
          stride(kChunk * sides), own(to - from), begin(from),
          end(min(to, (tile.count + kChunk - 1) / kChunk * kChunk)) {
        if (first < end) load_residual(first);
    }
    // row of the output and columns left, for this lane's first column of a chunk
    __device__ __forceinline__ int column() const { return GATED ? lane & 3 : lane & 1; }
    __device__ __forceinline__ int left(int c0) const {
        return f.any ? t.count - c0 - column() : 0;
    }
    __device__ __forceinline__ void load_residual(int c0) {
        if constexpr (!GATED) {
            if (f.g.residual && f.vec) {
                const int64_t M = f.g.M;
                const uint16_t *p = f.g.residual + (t.row0 + c0 + column()) * M + f.m;
                const int n = left(c0);
#pragma unroll
                for (int k = 0; k < kChunk / 2; ++k, p += 2 * M)
                    next[k] = 2 * k < n ? *reinterpret_cast<const uint32_t *>(p) : 0u;
            }
        }
    }
};

// Where the sums of k's other parts have TMEM lane `lane` of column c: neither
// lanes by columns (the sender, and finish_tile) nor fragments meet in a bank.
__device__ __forceinline__ int sum_lane(int lane, int c) { return lane ^ ((c >> 1 & 3) << 3); }

// The part out of TMEM; arrives on `done` (0: nowhere) once it has read its
// columns.  parts > 0: so many other parts' sums of these columns are in
// `sums`.  Lanes swap values so that each holds two adjacent features of one
// column; bias, activation, residual and stores then run as loops over the
// chunk, with nothing to decide per value, so their latencies overlap
// (deciding per pair took 22 us per 256 x 256 tile, now about 3).
template <bool GATED>
__device__ __forceinline__ void finish_tile(TilePart<GATED> &part, uint32_t tmem, uint32_t done,
                                            const float *sums, int parts) {
    const Finish<GATED> &f = part.f;
    const Gemm &g = f.g;
    const Tile &t = part.t;
    const int lane = part.lane, own = part.own, begin = part.begin, end = part.end;
    const int quarter = part.quarter, stride = part.stride;
    const bool odd = lane & 1, upper = lane & 2;
    const int64_t M = g.M;
    if (part.first >= end) {            // nothing for this warp
        if (done && lane == 0) bar_arrive(done);
        return;
    }
#pragma unroll 1
    for (int c0 = part.first; c0 < end; c0 += stride) {
        const int64_t row = t.row0 + c0 + part.column();
        const int left = part.left(c0);
        uint32_t r[kChunk];
        tmem_load16(tmem + c0, r);
        if (done && c0 + stride >= end) {       // the accumulator has been read
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(done);
        }
        uint32_t res[GATED ? 1 : kChunk / 2];
        if constexpr (!GATED) {
#pragma unroll
            for (int k = 0; k < kChunk / 2; ++k) res[k] = part.next[k];
        }
        if (c0 + stride < end) part.load_residual(c0 + stride);
        for (int k = 0; k < parts; ++k) {
            const float *from = sums + (k * own + c0 - begin) * 128 + quarter * 32;
#pragma unroll
            for (int c = 0; c < kChunk; ++c)
                r[c] = __float_as_uint(__uint_as_float(r[c]) + from[c * 128 + sum_lane(lane, c)]);
        }
        if constexpr (GATED) {
            float gate[kChunk / 2], up[kChunk / 2];     // [2k], [2k + 1]: features f, f + 1,
#pragma unroll                                          // column 4k
            for (int k = 0; k < kChunk / 4; ++k) {
                // neighbours: (gate, up) of columns 4k + odd and 4k + 2 + odd
                float a[2], u[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float lo = __uint_as_float(r[4 * k + 2 * j]);
                    const float hi = __uint_as_float(r[4 * k + 2 * j + 1]);
                    const float v = __shfl_xor_sync(0xFFFFFFFFu, odd ? lo : hi, 1);
                    a[j] = odd ? v : lo;
                    u[j] = odd ? hi : v;
                }
                // the next feature's: lanes with `upper` keep the second column
                const float va = __shfl_xor_sync(0xFFFFFFFFu, upper ? a[0] : a[1], 2);
                const float vu = __shfl_xor_sync(0xFFFFFFFFu, upper ? u[0] : u[1], 2);
                gate[2 * k] = (upper ? va : a[0]) + f.bias[0];
                gate[2 * k + 1] = (upper ? a[1] : va) + f.bias[1];
                up[2 * k] = (upper ? vu : u[0]) + f.bias[GATED ? 2 : 0];
                up[2 * k + 1] = (upper ? u[1] : vu) + f.bias[GATED ? 3 : 1];
            }
            if (!f.vec) {
#pragma unroll
                for (int k = 0; k < kChunk / 4; ++k)
                    if (4 * k < left)
                        finish_scalar<true>(g, f.m, row + 4 * k, gate[2 * k], gate[2 * k + 1],
                                            up[2 * k], up[2 * k + 1]);
                continue;
            }
            if (g.preact) {
                uint16_t *p = g.preact + row * 2 * M + f.m;
#pragma unroll
                for (int k = 0; k < kChunk / 4; ++k, p += 8 * M)
                    if (4 * k < left) {
                        store2(p, gate[2 * k], gate[2 * k + 1]);
                        store2(p + M, up[2 * k], up[2 * k + 1]);
                    }
            }
            act_all(gate, g.act);
            uint16_t *p = static_cast<uint16_t *>(g.out) + row * M + f.m;
#pragma unroll
            for (int k = 0; k < kChunk / 4; ++k, p += 4 * M)
                if (4 * k < left) store2(p, gate[2 * k] * up[2 * k],
                                         gate[2 * k + 1] * up[2 * k + 1]);
        } else {
            float z[kChunk];                // [2k], [2k + 1]: features m, m + 1, column 2k
#pragma unroll
            for (int k = 0; k < kChunk / 2; ++k) {
                const float lo = __uint_as_float(r[2 * k]), hi = __uint_as_float(r[2 * k + 1]);
                const float v = __shfl_xor_sync(0xFFFFFFFFu, odd ? lo : hi, 1);
                z[2 * k] = (odd ? v : lo) + f.bias[0];
                z[2 * k + 1] = (odd ? hi : v) + f.bias[1];
            }
            if (!f.vec) {
#pragma unroll
                for (int k = 0; k < kChunk / 2; ++k)
                    if (2 * k < left)
                        finish_scalar<false>(g, f.m, row + 2 * k, z[2 * k], z[2 * k + 1], 0.f, 0.f);
                continue;
            }
            const int64_t at = row * M + f.m;
            if (g.preact) {
                uint16_t *p = g.preact + at;
#pragma unroll
                for (int k = 0; k < kChunk / 2; ++k, p += 2 * M)
                    if (2 * k < left) store2(p, z[2 * k], z[2 * k + 1]);
            }
            act_all(z, g.act);
            if (g.residual) {
#pragma unroll
                for (int k = 0; k < kChunk / 2; ++k) {
                    z[2 * k] += bf16_lo(res[k]);
                    z[2 * k + 1] += bf16_hi(res[k]);
                }
            }
            if (g.out_f32) {
                float *p = static_cast<float *>(g.out) + at;
#pragma unroll
                for (int k = 0; k < kChunk / 2; ++k, p += 2 * M)
                    if (2 * k < left)
                        *reinterpret_cast<float2 *>(p) = make_float2(z[2 * k], z[2 * k + 1]);
            } else {
                uint16_t *p = static_cast<uint16_t *>(g.out) + at;
#pragma unroll
                for (int k = 0; k < kChunk / 2; ++k, p += 2 * M)
                    if (2 * k < left) store2(p, z[2 * k], z[2 * k + 1]);
            }
        }
    }
}

// The same where rows are whole 16-byte pieces, which is nearly always.  The
// chunk comes as fragments of 8 x 8 matrices, is finished as it is, packed in
// pairs of columns, and transposed through the warp's stash into 16-byte pieces of
// rows: a third of the instructions, which is what the other form is bound by
// (4096 x 4864 x 64: 14.5 us there, 11.2 here; gated 13.7 and 10.6).
template <bool GATED, bool RESIDUAL>
struct WidePart {
    const Gemm &g;
    const Tile t;
    int lane, quarter, first, stride, own, begin, end, m;
    float bias[4];                      // of the features this thread has (gated: gate, up, ...)
    uint4 next[RESIDUAL ? 2 : 1];       // residual pieces of the next chunk
    static constexpr int kPieces = GATED ? 2 : 4;       // of a row

    __device__ __forceinline__ WidePart(const Gemm &gemm, const Tile &tile, int m_cta,
                                        int warp_quarter, int side, int sides, int warp_lane,
                                        int from, int to)
        : g(gemm), t(tile), lane(warp_lane), quarter(warp_quarter), first(from + kChunk * side),
          stride(kChunk * sides), own(to - from), begin(from),
          end(min(to, (tile.count + kChunk - 1) / kChunk * kChunk)),
          m(m_cta + warp_quarter * 8 * kPieces) {
        const uint16_t *b = g.bias + static_cast<int64_t>(t.e) * (GATED ? 2 : 1) * g.M;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int feature = m + 8 * (GATED ? i >> 1 : i) + (lane >> 2);
            bias[i] = g.bias && feature < g.M
                          ? bf16_value(b, GATED && (i & 1) ? g.M + feature : feature) : 0.f;
        }
        if (first < end) load_residual(first);
        // the other chunks into L2, a row a lane (4096 x 4864 x 64: 24.7 -> 22.8 us)
        if constexpr (RESIDUAL) {
            const int row = lane & 15;
            if (m < g.M)
                for (int c0 = first + (lane < 16 ? 1 : 2) * stride; c0 < end; c0 += 2 * stride)
                    if (c0 + row < t.count)
                        prefetch_l2(g.residual + (t.row0 + c0 + row) * g.M + m);
        }
    }
    // this thread's piece p of a chunk: its token, or -1 where there is none
    __device__ __forceinline__ int token(int p, int c0) const {
        const int n = 8 * p + lane / kPieces;
        return c0 + n < t.count && m + 8 * (lane % kPieces) < g.M ? n : -1;
    }
    __device__ __forceinline__ int64_t at(int c0, int n, int64_t pitch) const {
        return (t.row0 + c0 + n) * pitch + m + 8 * (lane % kPieces);
    }
    __device__ __forceinline__ void load_residual(int c0) {
        if constexpr (RESIDUAL) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int n = token(p, c0);
                next[p] = make_uint4(0, 0, 0, 0);
                if (n >= 0)
                    next[p] = *reinterpret_cast<const uint4 *>(g.residual + at(c0, n, g.M));
            }
        }
    }
    // stash offsets: row (token) and piece of matrix lane / 8, row lane % 8, and of
    // this thread's piece; swizzled so that eight rows, or pieces, meet no bank
    __device__ __forceinline__ uint32_t matrix_at(int u) const {
        if constexpr (GATED) {
            const int i = lane >> 3, row = 8 * (i >> 1) + (lane & 7);
            return row * 32 + (((i & 1) ^ (row >> 2 & 1)) << 4);
        } else {
            const int row = lane & 7;
            return u * 512 + row * 64 + (((lane >> 3) ^ (row >> 1)) << 4);
        }
    }
    __device__ __forceinline__ uint32_t piece_at(int p) const {
        if constexpr (GATED) return (lane >> 1) * 32 + (((lane & 1) ^ (lane >> 3 & 1)) << 4);
        else return p * 512 + (lane >> 2) * 64 + (((lane & 3) ^ (lane >> 3)) << 4);
    }
};

// A chunk of bf16 pairs (w[j][i]: columns 8 j .., features 8 i ..) to rows of p.
template <bool GATED, bool RESIDUAL>
__device__ __forceinline__ void store_chunk(const WidePart<GATED, RESIDUAL> &part, uint32_t stash,
                                            const uint32_t (&w)[2][GATED ? 2 : 4], int c0,
                                            uint16_t *p, int64_t pitch) {
    __syncwarp();               // the stash has been read
    if constexpr (GATED) {
        store_transposed(stash + part.matrix_at(0), w[0][0], w[0][1], w[1][0], w[1][1]);
    } else {
        store_transposed(stash + part.matrix_at(0), w[0][0], w[0][1], w[0][2], w[0][3]);
        store_transposed(stash + part.matrix_at(1), w[1][0], w[1][1], w[1][2], w[1][3]);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < (GATED ? 1 : 2); ++k) {
        const uint4 v = shared_load16(stash + part.piece_at(k));
        const int n = part.token(k, c0);
        if (n >= 0) *reinterpret_cast<uint4 *>(p + part.at(c0, n, pitch)) = v;
    }
}

template <bool GATED, bool RESIDUAL>
__device__ __forceinline__ void finish_wide(WidePart<GATED, RESIDUAL> &part, uint32_t stash,
                                            uint32_t tmem, uint32_t done, const float *sums,
                                            int parts) {
    const Gemm &g = part.g;
    const int lane = part.lane, end = part.end, stride = part.stride;
    if (part.first >= end) {            // nothing for this warp
        if (done && lane == 0) bar_arrive(done);
        return;
    }
#pragma unroll 1
    for (int c0 = part.first; c0 < end; c0 += stride) {
        uint32_t r[kChunk];
        tmem_load_fragments(tmem + c0, r);
        if (done && c0 + stride >= end) {       // the accumulator has been read
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(done);
        }
        uint32_t res[2][4];             // the residual, as fragments
        if constexpr (RESIDUAL) {
            __syncwarp();
#pragma unroll
            for (int p = 0; p < 2; ++p) shared_store16(stash + part.piece_at(p), part.next[p]);
            if (c0 + stride < end) part.load_residual(c0 + stride);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 2; ++j) load_transposed(stash + part.matrix_at(j), res[j]);
        }
        float z[2][4][2];               // [columns 8 j ..][features 8 i .., gated: gate, up][pair]
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    z[j][i][e] = __uint_as_float(r[8 * (i >> 1) + 4 * j + 2 * (i & 1) + e]);
        for (int k = 0; k < parts; ++k) {
            const float *from = sums + (k * part.own + c0 - part.begin) * 128 + part.quarter * 32;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = 8 * j + 2 * (lane & 3) + e;
                        z[j][i][e] += from[c * 128 + sum_lane(8 * i + (lane >> 2), c)];
                    }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) z[j][i][e] += part.bias[i];
        if constexpr (GATED) {
            uint32_t w[2][2];
            if (g.preact) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            w[j][i] = pack_bf16x2(z[j][2 * i + h][0], z[j][2 * i + h][1]);
                    store_chunk(part, stash, w, c0,
                                      g.preact + static_cast<int64_t>(h) * g.M,
                                      2 * static_cast<int64_t>(g.M));
                }
            }
            float a[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) a[k] = z[k >> 2][k & 2][k & 1];
            act_all(a, g.act);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    w[j][i] = pack_bf16x2(a[4 * j + 2 * i] * z[j][2 * i + 1][0],
                                          a[4 * j + 2 * i + 1] * z[j][2 * i + 1][1]);
            store_chunk(part, stash, w, c0, static_cast<uint16_t *>(g.out), g.M);
        } else {
            uint32_t w[2][4];
            if (g.preact) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[j][i] = pack_bf16x2(z[j][i][0], z[j][i][1]);
                store_chunk(part, stash, w, c0, g.preact, g.M);
            }
            float a[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) a[k] = z[k >> 3][k >> 1 & 3][k & 1];
            act_all(a, g.act);
            if constexpr (RESIDUAL) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[8 * j + 2 * i] += bf16_lo(res[j][i]);
                        a[8 * j + 2 * i + 1] += bf16_hi(res[j][i]);
                    }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[j][i] = pack_bf16x2(a[8 * j + 2 * i], a[8 * j + 2 * i + 1]);
            store_chunk(part, stash, w, c0, static_cast<uint16_t *>(g.out), g.M);
        }
    }
}

// k in parts: the columns of a tile are shared out over the parts, kChunk at a
// time, and each part sends its sums of the others' columns into their shared
// memory, [sender][column][128 rows of A].
__host__ __device__ __forceinline__ int own_columns(int bn, int split) {
    return ((bn + split - 1) / split + kChunk - 1) / kChunk * kChunk;
}

// Shared memory for the other parts' sums.
constexpr int kMaxReceived = 64 * 1024;

__host__ __device__ __forceinline__ int received_bytes(int bn, int split) {
    return (split - 1) * own_columns(bn, split) * 512;
}

template <int CG>
__device__ __forceinline__ void send_columns(const Tile &t, uint32_t tmem, uint32_t buf, int split,
                                             int part, int rank0, int quarter, int side, int sides,
                                             int lane) {
    const int own = own_columns(t.bn, split);
    for (int c0 = kChunk * side; c0 < t.count; c0 += kChunk * sides) {
        const int owner = c0 / own;
        if (owner == part) continue;
        uint32_t r[kChunk];
        tmem_load16(tmem + c0, r);
        const int slot = part < owner ? part : part - 1;
        const uint32_t at = map_rank(
            buf + ((slot * own + c0 - owner * own) * 128 + quarter * 32) * 4, rank0 + owner * CG);
#pragma unroll
        for (int c = 0; c < kChunk; ++c)
            store_remote(at + (c * 128 + sum_lane(lane, c)) * 4, r[c]);
    }
}

// --------------------------------------------------------------- kernel

// Expert groups (all threads): their rows, clipped to the buffer, the width of
// the column tiles, from the largest group, the tiles before each expert, and
// the parts of k: as many as the launch's clusters have room for while each
// halving saves more k blocks (400 clocks) than it costs to join.
template <int CG>
__device__ __forceinline__ void count_tiles(const Gemm &g, const TcPlan &p, Header *h) {
    const int lane = threadIdx.x & 31;
    int most = 0;
    for (int e = threadIdx.x; e < g.E; e += kTcThreads) {
        const int first = g.offsets[e], rows = g.counts[e];
        const int count = first < 0 ? 0 : max(0, min(rows, g.N - first));
        h->first[e] = first;
        h->count[e] = count;
        most = max(most, count);
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) h->prefix[threadIdx.x / 32] = most;      // until the scan below
    __syncthreads();
    if (threadIdx.x >= 32) return;
    most = __reduce_max_sync(0xFFFFFFFFu, lane < kTcThreads / 32 ? h->prefix[lane] : 0);
    const int bn = max(1, (min(most, p.bn) + 16 * CG - 1) / (16 * CG)) * 16 * CG;
    int before = 0;
    for (int e0 = 0; e0 < g.E; e0 += 32) {
        const int e = e0 + lane;
        const int v = e < g.E && h->count[e] > 0 ? (h->count[e] - 1) / bn + 1 : 0;
        int sum = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += w;
        }
        __syncwarp();
        if (e < g.E) h->prefix[e] = before + sum - v;
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (lane == 0) {
        const int tiles = before * p.m_tiles, units = gridDim.x / CG;
        int blocks = steps_of(g.K, kBlockK), log = 0;
        while (log < p.log_split && tiles <= units >> (log + 1) &&
               received_bytes(bn, 2 << log) <= kMaxReceived &&
               (blocks /= 2) * 400 > (log ? 300 << log : 1500 + 10 * bn))
            ++log;
        h->prefix[g.E] = before;
        h->bn = bn;
        h->tiles = tiles;
        h->log_split = log;
    }
}

template <int CG, bool GATED, int N>
__global__ void __launch_bounds__(kTcThreads, 1)
gemm_tc_kernel(const __grid_constant__ Work<N> work) {
    static_assert(N == 1 || (CG == 2 && !GATED), "two products run on pairs, without k in parts");
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = (smem_addr(smem) + 1023) & ~1023u;
    Header *h = reinterpret_cast<Header *>(smem + (base - smem_addr(smem)));
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    // the CTA's place in its cluster: which unit, and which half of a pair
    const bool clustered = N == 1 && work.p[0].log_split > 0;
    const int rank = CG == 2 || clustered ? static_cast<int>(cluster_rank()) : 0;
    const int unit = rank / CG, half = rank % CG, lead = unit * CG;
    const bool leader = half == 0;
    const uint16_t pair = static_cast<uint16_t>(3 << lead);
    volatile int *gave_up = &h->gave_up;
    // the warps that finish tiles, two for each quarter of the lanes, or three with
    // those that have no rows to gather: a warp may read the TMEM lanes of its
    // number modulo 4
    const bool gathers = N == 1 && work.p[0].gather;
    const int sides = gathers ? 2 : 3, quarter = warp & 3;
    const int side = warp >= 2 && warp < kCopyWarp ? (warp - 2) >> 2
                     : !gathers && warp > kBiasWarp ? 2 : -1;
    // expert groups: the tiles follow from what the previous kernels wrote
    const bool grouped = N == 1 && work.g[0].E;

    if (threadIdx.x == 0) {
        for (int i = 0; i < N; ++i) {
            prefetch_map(&work.map[i][0]);
            prefetch_map(&work.map[i][1]);
        }
        for (int i = 0; i < kMaxStages; ++i) {
            bar_init(smem_addr(&h->full[i]), 1);
            bar_init(smem_addr(&h->empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_addr(&h->acc_full[i]), 1);
            bar_init(smem_addr(&h->acc_empty[i]), 4 * sides * CG);
        }
        h->gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<CG>(smem_addr(&h->tmem), 2 * kMaxBn);
    if (grouped) {
        wait_previous_kernel();
        allow_next_kernel();
        count_tiles<CG>(work.g[0], work.p[0], h);
    }
    fence_before();
    if (CG == 2) {
        cluster_sync();
    } else {
        if (clustered) cluster_arrive();        // awaited before the first remote store
        __syncthreads();
    }
    fence_after();

    const uint32_t tmem = h->tmem;
    int tiles, bn_max, log_split = 0, bytes_received = 0;
    if (grouped) {
        tiles = h->tiles;
        bn_max = h->bn;
        log_split = h->log_split;
        bytes_received = received_bytes(bn_max, 1 << log_split);
    } else {
        if (N == 1) {
            log_split = work.p[0].log_split;
            bytes_received = work.p[0].received;
        }
        tiles = work.p[0].n_tiles * work.p[0].m_tiles;
        bn_max = work.p[0].bn;
        if constexpr (N == 2) {
            tiles += work.p[1].n_tiles * work.p[1].m_tiles;
            bn_max = max(bn_max, work.p[1].bn);
        }
    }
    // the epilogue warps' stashes, the other parts' sums, the stages
    const uint32_t stash = base + kHeader - (grouped ? 0 : kStashes) +
                           (4 * side + quarter) * kStash;
    const uint32_t received = base + kHeader + (grouped ? kStashes : 0);
    const uint32_t stage0 = received + bytes_received;
    const int split = 1 << log_split, part = unit & (split - 1);
    const int bnc_max = bn_max / CG;                // B rows per CTA
    // transposed B comes in blocks of 64 columns; a multiple of 2048 bytes
    const bool any_mn = work.g[0].b_mn || work.g[N - 1].b_mn;
    const uint32_t b_bytes = (any_mn ? (bnc_max + 63) / 64 * 64 : bnc_max) * kBlockK * 2;
    const uint32_t stage_bytes = kATile + b_bytes;
    const int stages = min(static_cast<unsigned>(kMaxStages),
                           (base + kHeader + kStageArea - stage0) / stage_bytes);
    const int first_tile = (blockIdx.x / CG) >> log_split;
    const int step = (gridDim.x / CG) >> log_split;     // k in parts: at least as many as tiles
    const int m_cta_rows = GATED ? 64 : 128;        // features per CTA
    // the product that a tile belongs to, and this part's k blocks of it
    auto product_of = [&](int ti) { return N == 2 && ti >= work.tiles0 ? 1 : 0; };
    auto tile_of = [&](int ti, int q) {
        return tile_at<CG, GATED>(work.g[q], work.p[q], h, q ? ti - work.tiles0 : ti);
    };
    auto k_range = [&](int q, int *kb0, int *kb1) {
        const int blocks = steps_of(work.g[q].K, kBlockK);
        *kb0 = (blocks * part) >> log_split;        // blocks <= 2^25, part < 16
        *kb1 = (blocks * (part + 1)) >> log_split;
    };
    auto wait_for_tile = [&](int n, int q) {
        int kb0, kb1;
        k_range(q, &kb0, &kb1);
        const bool ok = wait(smem_addr(&h->acc_full[n & 1]), (n >> 1) & 1, gave_up, kb1 - kb0);
        return __all_sync(0xFFFFFFFFu, ok);
    };
    // Launched as a dependent of the previous kernel on the stream: everything
    // up to a role's first tile comes from the parameters, and global memory is
    // touched behind this.
    auto begin = [&](int ti) {
        if (ti == first_tile && !grouped) wait_previous_kernel();
    };

    if (warp == 0) {
        // ---- copies of A, and the stages' byte counts
        if (elect_one()) {
            int s = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int ti = first_tile; ti < tiles && ok; ti += step) {
                const int q = product_of(ti);
                const Gemm &g = work.g[q];
                const TcPlan &p = work.p[q];
                const CUtensorMap *map = &work.map[q][0];
                const Tile t = tile_of(ti, q);
                int kb0, kb1;
                k_range(q, &kb0, &kb1);
                const int bnc = t.bn / CG, m0 = t.m0 + half * m_cta_rows;
                const uint32_t b_tx = p.gather ? bnc * 128u
                                      : g.b_mn ? (bnc + 63) / 64 * 8192u
                                               : (bnc + p.box_rows - 1) / p.box_rows *
                                                     p.box_rows * 128u;
                const uint32_t tx = CG * (kATile + b_tx);
                begin(ti);
                if (ti == first_tile) allow_next_kernel();
                auto blocks_of = [&](auto copy) {
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!wait(smem_addr(&h->empty[s]), phase, gave_up)) return false;
                        const uint32_t full = smem_addr(&h->full[s]);
                        if (leader) bar_expect(full, tx);
                        copy(stage0 + s * stage_bytes, kb * kBlockK,
                             CG == 2 ? map_rank(full, lead) : full);
                        if (++s == stages) { s = 0; phase ^= 1; }
                    }
                    return true;
                };
                if (g.a_mn)
                    ok = blocks_of([&](uint32_t a, int k, uint32_t bar) {
                        tma_2d<CG>(a, map, m0, k, bar);
                        tma_2d<CG>(a + 8192, map, m0 + 64, k, bar);
                    });
                else if (GATED && p.vectors)
                    ok = blocks_of([&](uint32_t a, int k, uint32_t bar) {
                        tma_5d<CG>(a, map, k, 0, 0, m0 >> 3, t.e, bar);
                    });
                else
                    ok = blocks_of([&](uint32_t a, int k, uint32_t bar) {
                        tma_4d<CG>(a, map, k, 0, m0, t.e, bar);
                    });
            }
            // every stage handed back: no copy or arrival is left in flight
            for (int i = 0; i < stages; ++i) {
                if (!wait(smem_addr(&h->empty[s]), phase, gave_up)) break;
                if (++s == stages) { s = 0; phase ^= 1; }
            }
            if (*gave_up)       // copies still in flight land before the CTA leaves
                for (const long long begin = clock64(); clock64() - begin < 2000000;)
                    __nanosleep(1000);
        }
    } else if (warp >= kCopyWarp && side < 0) {
        // ---- copies of B: one lane, or some of each warp when rows are gathered
        int s = 0;
        uint32_t phase = 1;
        if (gathers) {
            const Gemm &g = work.g[0];
            int kb0, kb1;
            k_range(0, &kb0, &kb1);
            const int quad = (warp - kCopyWarp) * kGatherLanes + lane;      // of rows
            for (int ti = first_tile; ti < tiles; ti += step) {
                const Tile t = tile_of(ti, 0);
                const int bnc = t.bn / CG;
                int4 rows = make_int4(-1, -1, -1, -1);      // -1: a row of zeros
                const bool mine = lane < kGatherLanes && 4 * quad < bnc;
                if (mine) {
                    const int valid = t.count - half * bnc - 4 * quad;
                    const int32_t *at = g.row_token + t.row0 + half * bnc + 4 * quad;
                    if (valid > 0) rows.x = at[0];
                    if (valid > 1) rows.y = at[1];
                    if (valid > 2) rows.z = at[2];
                    if (valid > 3) rows.w = at[3];
                }
                bool ok = true;
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = wait(smem_addr(&h->empty[s]), phase, gave_up);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const uint32_t full = smem_addr(&h->full[s]);
                    if (mine)
                        tma_gather4<CG>(stage0 + s * stage_bytes + kATile + quad * 512,
                                        &work.map[0][1],
                                        kb * kBlockK, rows, CG == 2 ? map_rank(full, lead) : full);
                    if (++s == stages) { s = 0; phase ^= 1; }
                }
                if (!ok) break;
            }
        } else if (warp > kCopyWarp) {
            // the bias gradient, 32 columns a CTA
            if (work.bias.dbias) {
                wait_previous_kernel();
                for (int c = blockIdx.x * 32; c < work.bias.cols; c += gridDim.x * 32)
                    sum_columns(work.bias, c + lane);
            }
        } else if (elect_one()) {
            bool ok = true;
            for (int ti = first_tile; ti < tiles && ok; ti += step) {
                const int q = product_of(ti);
                const Gemm &g = work.g[q];
                const TcPlan &p = work.p[q];
                const CUtensorMap *map = &work.map[q][1], *wide = &work.map[q][2];
                const Tile t = tile_of(ti, q);
                int kb0, kb1;
                k_range(q, &kb0, &kb1);
                const int bnc = t.bn / CG;
                const int row0 = static_cast<int>(t.row0 + half * bnc);
                const int rows = g.b_mn ? 64 : p.box_rows;      // of one copy
                const int boxes = (bnc + rows - 1) / rows;
                begin(ti);
                auto blocks_of = [&](auto copy) {
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!wait(smem_addr(&h->empty[s]), phase, gave_up)) return false;
                        const uint32_t full = smem_addr(&h->full[s]);
                        copy(stage0 + s * stage_bytes + kATile, kb * kBlockK,
                             CG == 2 ? map_rank(full, lead) : full);
                        if (++s == stages) { s = 0; phase ^= 1; }
                    }
                    return true;
                };
                if (g.b_mn)
                    ok = blocks_of([&](uint32_t b, int k, uint32_t bar) {
                        for (int i = 0; i < boxes; ++i)
                            tma_2d<CG>(b + i * 8192, map, row0 + i * 64, k, bar);
                    });
                else if (boxes == 1)
                    ok = blocks_of([&](uint32_t b, int k, uint32_t bar) {
                        tma_2d<CG>(b, map, k, row0, bar);
                    });
                else
                    ok = blocks_of([&](uint32_t b, int k, uint32_t bar) {
                        int at = 0;
                        if (p.wide_rows)
                            for (; at + p.wide_rows <= bnc; at += p.wide_rows)
                                tma_2d<CG>(b + at * 128, wide, k, row0 + at, bar);
                        for (; at < bnc; at += rows)
                            tma_2d<CG>(b + at * 128, map, k, row0 + at, bar);
                    });
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- products
        if (leader && elect_one()) {
            int s = 0, n = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int ti = first_tile; ti < tiles && ok; ti += step, ++n) {
                const int q = product_of(ti);
                const Gemm &g = work.g[q];
                const Tile t = tile_of(ti, q);
                int kb0, kb1;
                k_range(q, &kb0, &kb1);
                // D fp32, A and B bf16, transposes, N, M
                const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) |
                                       (static_cast<uint32_t>(g.a_mn) << 15) |
                                       (static_cast<uint32_t>(g.b_mn) << 16) |
                                       (static_cast<uint32_t>(t.bn >> 3) << 17) |
                                       (static_cast<uint32_t>(128 * CG >> 4) << 24);
                const uint32_t d = tmem + (n & 1) * kMaxBn;
                const uint32_t a_step = g.a_mn ? 2048 >> 4 : 32 >> 4;
                const uint32_t b_step = g.b_mn ? 2048 >> 4 : 32 >> 4;
                begin(ti);      // or the previous kernel's time counts as a copy's
                if (!wait(smem_addr(&h->acc_empty[n & 1]), ((n >> 1) & 1) ^ 1, gave_up)) break;
                fence_after();
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wait(smem_addr(&h->full[s]), phase, gave_up)) { ok = false; break; }
                    fence_after();
                    const uint32_t a = stage0 + s * stage_bytes;
                    const uint64_t da = smem_desc(a, g.a_mn);
                    const uint64_t db = smem_desc(a + kATile, g.b_mn);
#pragma unroll
                    for (int k = 0; k < kBlockK / 16; ++k)
                        mma_bf16<CG>(d, da + k * a_step, db + k * b_step, idesc,
                                     kb > kb0 || k > 0);
                    mma_commit<CG>(smem_addr(&h->empty[s]), pair);
                    if (++s == stages) { s = 0; phase ^= 1; }
                }
                if (ok) mma_commit<CG>(smem_addr(&h->acc_full[n & 1]), pair);
            }
        }
    } else {
        // ---- epilogue
        int n = 0;
        for (int ti = first_tile; ti < tiles; ti += step, ++n) {
            const int q = product_of(ti);
            const Tile t = tile_of(ti, q);
            const uint32_t acc = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                 (n & 1) * kMaxBn;
            begin(ti);
            if (split > 1) {        // joined below
                (void)wait_for_tile(n, q);
                fence_after();
                break;
            }
            const uint32_t done = map_rank(smem_addr(&h->acc_empty[n & 1]),
                                           CG == 2 ? lead : cluster_rank());
            auto finish = [&](auto &part_of, auto out_of_tmem) {
                if (!wait_for_tile(n, q)) return false;
                fence_after();
                out_of_tmem(part_of);
                return true;
            };
            const int m0 = t.m0 + half * m_cta_rows;
            bool ok;
            auto wide = [&](auto &w) { finish_wide(w, stash, acc, done, nullptr, 0); };
            if (work.p[q].vectors && !GATED && work.g[q].residual) {
                WidePart<GATED, !GATED> part_of(work.g[q], t, m0, quarter, side, sides, lane, 0,
                                                t.bn);
                ok = finish(part_of, wide);
            } else if (work.p[q].vectors) {
                WidePart<GATED, false> part_of(work.g[q], t, m0, quarter, side, sides, lane, 0,
                                               t.bn);
                ok = finish(part_of, wide);
            } else {
                TilePart<GATED> part_of(work.g[q], t, m0, quarter, side, sides, lane, 0, t.bn);
                ok = finish(part_of, [&](auto &w) {
                    finish_tile<GATED>(w, acc, done, nullptr, 0);
                });
            }
            if (!ok) break;
        }
    }
    __syncwarp();
    if (N == 1 && split > 1) {
        const uint32_t acc = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        if (CG == 1) cluster_wait();        // every part has started
        if (side >= 0 && first_tile < tiles) {
            const Tile t = tile_of(first_tile, 0);
            if (!*gave_up)
                send_columns<CG>(t, acc, received, split, part, (unit - part) * CG + half, quarter,
                                 side, sides, lane);
            const int own = own_columns(t.bn, split);
            const float *sums = reinterpret_cast<const float *>(smem + (received -
                                                                        smem_addr(smem)));
            const int m0 = t.m0 + half * m_cta_rows, from = part * own;
            if (work.p[0].vectors && !GATED && work.g[0].residual) {
                WidePart<GATED, !GATED> part_of(work.g[0], t, m0, quarter, side, sides, lane, from,
                                                from + own);
                cluster_sync();         // every part's sums have arrived
                if (!*gave_up) finish_wide(part_of, stash, acc, 0, sums, split - 1);
            } else if (work.p[0].vectors) {
                WidePart<GATED, false> part_of(work.g[0], t, m0, quarter, side, sides, lane, from,
                                               from + own);
                cluster_sync();
                if (!*gave_up) finish_wide(part_of, stash, acc, 0, sums, split - 1);
            } else {
                TilePart<GATED> part_of(work.g[0], t, m0, quarter, side, sides, lane, from,
                                        from + own);
                cluster_sync();
                if (!*gave_up) finish_tile<GATED>(part_of, acc, 0, sums, split - 1);
            }
        } else {
            cluster_sync();
        }
    }
    if (CG == 1 && clustered && split == 1) cluster_wait();
    fence_before();
    if (CG == 2) cluster_sync(); else __syncthreads();
    fence_after();
    if (warp == 1) tmem_free<CG>(tmem, 2 * kMaxBn);
}

// ----------------------------------------------------------------- host

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once (the library does not link
// the driver).
EncodeTiled encoder() {
    static EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

bool encode(CUtensorMap *map, const void *p, int rank, const cuuint64_t *dims,
            const cuuint64_t *strides, const cuuint32_t *box) {
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(p), dims,
                     strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int CG, bool GATED, int N>
cudaError_t start(const Work<N> &work, int64_t grid, cudaStream_t stream) {
    auto *kernel = gemm_tc_kernel<CG, GATED, N>;
    const int cluster = CG << (N == 1 ? work.p[0].log_split : 0);
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kSmemBytes);
    if (err == cudaSuccess && cluster > 8)
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, work);
}

// Clusters of 1, 2, 4, 8 and 16 CTAs with this kernel's shared memory that can
// run at once: SMs come in groups that a cluster does not span, so 152 SMs
// hold 36 clusters of 4, 15 of 8 and 7 of 16.  Asked once per device.
struct Slots {
    int n[5];
};

int ask_active_clusters(int size, int num_sms) {
    auto *kernel = gemm_tc_kernel<1, false, 1>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(size), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        n = num_sms / size > 1 ? num_sms / size / 2 : 1;
    }
    return n;
}

Slots cluster_slots(int num_sms) {
    static std::atomic<int> cache[kMaxDevices][5];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) dev = 0;
    Slots s = {{num_sms, num_sms / 2, 0, 0, 0}};
    for (int i = 2; i < 5; ++i) {
        s.n[i] = cache[dev][i].load(std::memory_order_relaxed);
        if (s.n[i] > 0) continue;
        s.n[i] = ask_active_clusters(1 << i, num_sms);
        cache[dev][i].store(s.n[i], std::memory_order_relaxed);
    }
    return s;
}

// One CTA or a pair per tile, columns per tile, parts of k.
struct Cut {
    int cg, bn, split;
};

// How a product that is not grouped is cut: one CTA or a pair per tile, columns
// per tile, parts of k.  Every choice is priced in SM clocks and the cheapest
// taken.  The figures are fits to sweeps over 17..4096 rows:
//   - a 64-deep k block takes the MMAs (2.7 clocks a column, 2.35 on a pair,
//     which reads half of B), the copies (80 bytes a clock into a single SM, 72
//     into each of a pair), the issue of both (290 clocks) or the latency of a
//     copy (2000) shared by the stages in flight, whichever is longest;
//   - a tile costs 300 clocks more, and its epilogue 800 and 13 a column, under
//     the next tile's products except for the last one; joining k's parts 2500
//     (pairs 4500), 300 a part and 30 a column; pairs 1800 for their barriers;
//   - HBM delivers 3580 bytes a clock; the shorter of its time and the SMs'
//     counts 15 %.
// Examples: 512 x 4096 x 7168 (gated) runs as 64 pairs of 128 columns, 24 us,
// against 29 us with 256 columns and k in two parts; 300 x 256 x 7168 as 80
// tiles of 64 columns and an eighth of k, 8.2 us, against 20 us unsplit.

// Bytes of a CTA's k block of both operands.
int block_bytes(const Gemm &g, int cg, int bn) {
    const int columns = bn / cg;
    return kATile + (g.b_mn ? (columns + 63) / 64 * 64 : columns) * 128;
}

// Clocks of one k block of a tile.
double block_clocks(const Gemm &g, int cg, int bn, int received) {
    const int bytes = block_bytes(g, cg, bn);
    const double copies = bytes / (cg == 1 ? 80.0 : 72.0);
    const double latency = 2000.0 / ((kStageArea - received) / bytes);
    const double mma = (cg == 1 ? 2.7 : 2.35) * bn;
    double clocks = mma > 290.0 ? mma : 290.0;
    if (copies > clocks) clocks = copies;
    return latency > clocks ? latency : clocks;
}

double epilogue_clocks(int bn) { return 800.0 + 13.0 * bn; }

// Tiles of at most `most` columns, evened out.
int even_columns(const Gemm &g, int cg, int most) {
    const int unit = 16 * cg;
    return static_cast<int>(ceil_div(ceil_div(g.N, ceil_div(g.N, most)), unit)) * unit;
}

Cut choose_cut(const Gemm &g, int64_t a_rows, const Slots &slots_of, double *price) {
    const int64_t blocks = ceil_div(g.K, kBlockK);
    const double hbm = 2.0 * (static_cast<double>(a_rows) * g.K +
                              static_cast<double>(g.N) * g.K +
                              static_cast<double>(g.N) * g.M) / 3580.0;
    Cut best = {2, kMaxBn, 1};
    *price = 1e300;
    for (int cg = 1; cg <= 2; ++cg) {
        const int64_t m_tiles = ceil_div(a_rows, 128 * cg);
        int64_t last = 0;
        for (int most = 32; most <= kMaxBn; most += 32) {
            const int64_t n_tiles = ceil_div(g.N, most);
            if (n_tiles == last) continue;
            last = n_tiles;
            const int bn = even_columns(g, cg, most);
            const int64_t tiles = m_tiles * n_tiles;
            for (int log = 0; cg << log <= 16 && 1 << log <= blocks; ++log) {
                const int split = 1 << log, slots = slots_of.n[log + cg - 1];
                const int received = received_bytes(bn, split);
                if (split > 1 && (tiles > slots || received > kMaxReceived)) break;
                const double tail = split == 1 ? epilogue_clocks(bn)
                                    : cg == 1  ? 2500.0 + 300.0 * split + 30.0 * bn
                                               : 4500.0 + 300.0 * split + 30.0 * bn;
                double tile = static_cast<double>(ceil_div(blocks, split)) *
                              block_clocks(g, cg, bn, received);
                if (split == 1 && tail > tile) tile = tail;
                double cost = static_cast<double>(ceil_div(tiles, slots)) * (tile + 300.0);
                cost = cost < hbm ? hbm + 0.15 * cost : cost + 0.15 * hbm;
                cost += tail + (cg == 2 ? 1800.0 : 0.0);
                if (cost < *price) {
                    *price = cost;
                    best = {cg, bn, split};
                }
            }
        }
    }
    return best;
}

// The same for two products in one launch, on pairs without k in parts: the
// tiles go round the pairs one by one, the first product's before the second's.
// The stages are as large as the larger product's; a product with one tile of
// columns shares no operand between its tiles and waits for HBM, 4000 clocks, in
// the fewer stages (12 x 4736 x 5192: both gradients 42 us in one launch, 33 in
// two).
double choose_two(const Gemm *g, int num_sms, int *bn) {
    const int pairs = num_sms / 2;
    auto product_clocks = [](const Gemm &p, int columns, int bytes) {
        const double latency = (p.N <= columns ? 4000.0 : 2000.0) / (kStageArea / bytes);
        const double clocks = block_clocks(p, 2, columns, 0);
        return ceil_div(p.K, kBlockK) * (latency > clocks ? latency : clocks);
    };
    double least = 1e300;
    for (int a = 64; a <= kMaxBn; a += 32) {
        const int bn0 = even_columns(g[0], 2, a);
        const int bytes0 = block_bytes(g[0], 2, bn0);
        const double tail0 = epilogue_clocks(bn0);
        const int64_t n0 = ceil_div(g[0].M, 256) * ceil_div(g[0].N, bn0);
        for (int b = 64; b <= kMaxBn; b += 32) {
            const int bn1 = even_columns(g[1], 2, b);
            const int bytes1 = block_bytes(g[1], 2, bn1), bytes = bytes0 > bytes1 ? bytes0 : bytes1;
            const double time0 = product_clocks(g[0], bn0, bytes);
            const double time1 = product_clocks(g[1], bn1, bytes);
            const double tail1 = epilogue_clocks(bn1);
            const double unit0 = 300.0 + (time0 > tail0 ? time0 : tail0);
            const double unit1 = 300.0 + (time1 > tail1 ? time1 : tail1);
            const int64_t n1 = ceil_div(g[1].M, 256) * ceil_div(g[1].N, bn1);
            // the pairs at the ends of the last rounds have the most to do
            const int64_t ends[4] = {0, n0 % pairs, (n0 + n1 + pairs - 1) % pairs, pairs - 1};
            double most = 0.0;
            for (int64_t j : ends) {
                const int64_t c0 = j < n0 ? (n0 - 1 - j) / pairs + 1 : 0;
                const int64_t c = j < n0 + n1 ? (n0 + n1 - 1 - j) / pairs + 1 : 0;
                const double load = c0 * unit0 + (c - c0) * unit1;
                if (load > most) most = load;
            }
            most += 1800.0 + (tail0 > tail1 ? tail0 : tail1);
            if (most < least) {
                least = most;
                bn[0] = bn0;
                bn[1] = bn1;
            }
        }
    }
    return least;
}

// Expert groups, whose sizes only the device knows.  If there can be at most two
// tiles an SM (a tile per group, and one for each 128 rows), single CTAs in
// clusters of 4, or 8 if the most tiles leave room for that many parts of k: the
// device then cuts k as far as the tiles that there are leave units idle.
// One token, 2 of 8 experts of 1536 x 4096 (gated): 15.2 us, 20.9 by pairs
// without parts; 13 tokens, 8 of 8 experts of 320 x 5400: 18.6 and 28.8; 300
// tokens, 1 of 8 experts of 512 x 1024: 9.6 and 10.7.  Otherwise pairs, which
// read half of B each and have no SM left over (36 clusters of 4 fill 144 of
// 152): 1000 tokens, 8 of 64 experts of 512 x 2048: 57 us, 70 by clusters.
Cut choose_groups(const Gemm &g, const Slots &slots_of) {
    const int64_t groups = g.E < g.N ? g.E : g.N;
    const int64_t most = ceil_div(static_cast<int64_t>(g.M) * (g.gated ? 2 : 1), 128) *
                         (groups + g.N / 128);
    if (most > 2 * slots_of.n[0]) return {2, kMaxBn, 1};
    return {1, 128, most <= slots_of.n[3] ? 8 : 4};
}

bool can_copy(const Gemm &g) {
    return aligned16(g.a) && aligned16(g.b) && (g.a_mn ? g.M : g.K) % 8 == 0 &&
           g.b_pitch % 8 == 0 && encoder();
}

// Plan and tensor maps of one product; false when the driver refuses a map.
bool describe(const Gemm &g, const Cut &cut, TcPlan *plan, CUtensorMap *map) {
    TcPlan &p = *plan;
    p = {};
    const int rows_per_feature = g.gated ? 2 : 1;
    const int64_t a_rows = static_cast<int64_t>(g.M) * rows_per_feature;
    p.gather = g.row_token != nullptr;
    p.vectors = g.M % 8 == 0 && !g.out_f32 && aligned16(g.out) && aligned16(g.residual) &&
                aligned16(g.preact);
    while (1 << p.log_split < cut.split) ++p.log_split;
    p.received = received_bytes(cut.bn, cut.split);
    p.bn = cut.bn;
    p.m_tiles = static_cast<int>(ceil_div(a_rows, 128 * cut.cg));
    if (g.E) {
        p.box_rows = 16;
    } else {
        p.n_tiles = static_cast<int>(ceil_div(g.N, p.bn));
        p.box_rows = p.bn / cut.cg;
    }
    bool ok;
    if (g.a_mn) {
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(g.M), static_cast<cuuint64_t>(g.K)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(g.M) * 2};
        const cuuint32_t box[2] = {64, 64};
        ok = encode(&map[0], g.a, 2, dims, strides, box);
    } else if (g.gated && p.vectors) {
        // [E][M / 8][gate, up][8][K]
        const cuuint64_t row = static_cast<cuuint64_t>(g.K) * 2;
        const cuuint64_t dims[5] = {static_cast<cuuint64_t>(g.K), 8, 2,
                                    static_cast<cuuint64_t>(g.M / 8),
                                    static_cast<cuuint64_t>(g.E ? g.E : 1)};
        const cuuint64_t strides[4] = {row, row * g.M, row * 8, row * a_rows};
        const cuuint32_t box[5] = {kBlockK, 8, 2, 8, 1};
        ok = encode(&map[0], g.a, 5, dims, strides, box);
    } else {
        // [E][M][gate, up][K]: a copy of (k, both, features) interleaves the rows
        const cuuint64_t row = static_cast<cuuint64_t>(g.K) * 2;
        const cuuint64_t dims[4] = {static_cast<cuuint64_t>(g.K),
                                    static_cast<cuuint64_t>(rows_per_feature),
                                    static_cast<cuuint64_t>(g.M),
                                    static_cast<cuuint64_t>(g.E ? g.E : 1)};
        const cuuint64_t strides[3] = {row * g.M, row, row * a_rows};
        const cuuint32_t box[4] = {kBlockK, static_cast<cuuint32_t>(rows_per_feature),
                                   static_cast<cuuint32_t>(128 / rows_per_feature), 1};
        ok = encode(&map[0], g.a, 4, dims, strides, box);
    }
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(g.b_mn ? g.N : g.K),
                                static_cast<cuuint64_t>(g.b_mn ? g.K : g.b_rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(g.b_pitch) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(g.b_mn      ? 64
                                                           : p.gather ? 1
                                                                      : p.box_rows)};
    ok = ok && encode(&map[1], g.b, 2, dims, strides, box);
    map[2] = map[1];
    if (g.E && !p.gather) {     // ragged groups: wide copies first, narrow ones for the rest
        p.wide_rows = 64;
        const cuuint32_t wide[2] = {64, 64};
        ok = ok && encode(&map[2], g.b, 2, dims, strides, wide);
    }
    return ok;
}

}  // namespace

bool launch_gemm_tc(const Gemm &g, const BiasSum &bias, int num_sms, cudaStream_t stream,
                    cudaError_t *err) {
    if (!can_copy(g)) return false;
    double price;
    const Slots slots_of = cluster_slots(num_sms);
    const Cut cut = g.E ? choose_groups(g, slots_of)
                        : choose_cut(g, static_cast<int64_t>(g.M) * (g.gated ? 2 : 1), slots_of,
                                     &price);
    Work<1> work;
    work.g[0] = g;
    work.tiles0 = 0;
    work.bias = bias;
    if (!describe(g, cut, &work.p[0], work.map[0])) return false;
    const TcPlan &p = work.p[0];
    int64_t units = static_cast<int64_t>(p.m_tiles) * p.n_tiles << p.log_split;
    const int64_t slots = num_sms / cut.cg;
    if (g.E)        // as many clusters as can run at once: the device shares the tiles out
        units = static_cast<int64_t>(slots_of.n[p.log_split + cut.cg - 1]) << p.log_split;
    else if (p.log_split == 0 && units > slots)
        units = slots;
    const int64_t grid = cut.cg * units;
    if (cut.cg == 2)
        *err = g.gated ? start<2, true>(work, grid, stream) : start<2, false>(work, grid, stream);
    else
        *err = g.gated ? start<1, true>(work, grid, stream) : start<1, false>(work, grid, stream);
    return true;
}

bool launch_two_gemms_tc(const Gemm *g, const BiasSum &bias, int num_sms, cudaStream_t stream,
                         cudaError_t *err) {
    if (!can_copy(g[0]) || !can_copy(g[1])) return false;
    // longer tiles first; two launches cost the second one's start, about 5000
    // clocks, but each may be cut as suits it
    const Gemm *order[2] = {&g[0], &g[1]};
    if (g[1].K > g[0].K) {
        order[0] = &g[1];
        order[1] = &g[0];
    }
    Work<2> work;
    work.g[0] = *order[0];
    work.g[1] = *order[1];
    work.bias = bias;
    int bn[2];
    double apart[2];
    const double together = choose_two(work.g, num_sms, bn);
    const Slots slots_of = cluster_slots(num_sms);
    for (int i = 0; i < 2; ++i) (void)choose_cut(work.g[i], work.g[i].M, slots_of, &apart[i]);
    if (together > apart[0] + apart[1] + 5000.0) return false;
    for (int i = 0; i < 2; ++i)
        if (!describe(work.g[i], {2, bn[i], 1}, &work.p[i], work.map[i])) return false;
    work.tiles0 = work.p[0].m_tiles * work.p[0].n_tiles;
    const int64_t units = static_cast<int64_t>(work.tiles0) +
                          static_cast<int64_t>(work.p[1].m_tiles) * work.p[1].n_tiles;
    const int64_t slots = num_sms / 2;
    *err = start<2, false>(work, 2 * (units < slots ? units : slots), stream);
    return true;
}

cudaError_t read_lost_waits(unsigned *count) {
    const cudaError_t err = cudaDeviceSynchronize();    // the copy waits for its own stream only
    return err != cudaSuccess ? err : cudaMemcpyFromSymbol(count, lost_waits, sizeof(*count));
}

}  // namespace moef
