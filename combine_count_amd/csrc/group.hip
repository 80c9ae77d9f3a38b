// Grouping received rows by expert for gfx950: a stable counting sort of the
// (row, slot) pairs by expert.
//
// The windows are cut into tiles of about 2048 slots, one block each.  A
// segment is what is sorted together: all windows (rank >= 0, one PE's
// experts), or each window by itself (rank -1, window p by PE p's experts).
//   1  hist_kernel: every tile's slots per expert, into the scratch;
//   2  place_kernel: a block sums the earlier tiles' counts (its bases) and
//      all tiles' (the groups' starts) itself, ranks its own slots in order
//      and writes the entries.
// Bases come from sums, not from atomics, so the order is fixed.  Up to
// kGroupLocalSlots slots a block counts all tiles' slots itself and step 1
// falls away; with more than kGroupSelfWords words of counts the sums of step
// 2 would read too much in every block, and two scan launches between turn
// the counts into bases.  Bound by latency (a launch, loads behind loads):
// 8 windows x 128 rows x 8 slots 9.5 us, 8 x 4096 x 8 (1.6 MB) 12.2 us.
//
// The order of slots inside a tile: a wave takes its quarter of the tile 64
// slots at a time; the lanes with the same expert find each other by a ballot
// per bit of the expert index, a slot's rank is the number of such lanes
// below it, and a counter per (wave, expert) in LDS carries over.
#include "ops_internal.h"

namespace epdc {
namespace {

constexpr int kWaves = 4;

struct Tile {
    int32_t window, rows;   // valid rows of the tile
    int64_t slot0;          // flat index of its first slot
    int32_t slots, live;    // slots of the tile (all rows), of its valid rows
    int32_t firstExpert;    // the segment's experts are [firstExpert, firstExpert + Epr)
    int32_t segment, segTile0;
};

__device__ __forceinline__ Tile tile_of(const GroupParams &P, int32_t tile) {
    Tile t;
    t.window = tile / P.tilesPerWindow;
    const int32_t r0 = (tile - t.window * P.tilesPerWindow) * P.tileRows;
    const int32_t rows = min(P.tileRows, P.M - r0);
    int32_t count = P.M;
    if (P.recvCount) count = min(max(P.recvCount[t.window], 0), P.M);
    t.rows = min(max(count - r0, 0), rows);
    t.slot0 = ((int64_t)t.window * P.M + r0) * P.K;
    t.slots = rows * P.K;
    t.live = t.rows * P.K;
    t.firstExpert = (P.rank < 0 ? t.window : P.rank) * P.Epr;
    t.segment = P.rank < 0 ? t.window : 0;
    t.segTile0 = P.rank < 0 ? t.window * P.tilesPerWindow : 0;
    return t;
}

// The tile's slots threadIdx.x, + 256, ...: their expert in the segment, -1 for
// none; all requested before the first is looked at.
constexpr int kSlotsPerThread = kGroupTileSlots / (64 * kWaves);
__device__ __forceinline__ void load_experts(const GroupParams &P, const Tile &t, int32_t (&ex)[kSlotsPerThread]) {
#pragma unroll
    for (int j = 0; j < kSlotsPerThread; ++j) {
        const int32_t i = j * 256 + threadIdx.x;
        ex[j] = i < t.live ? P.expertIds[t.slot0 + i] - t.firstExpert : -1;
    }
#pragma unroll
    for (int j = 0; j < kSlotsPerThread; ++j)
        if ((uint32_t)ex[j] >= (uint32_t)P.Epr) ex[j] = -1;
}

// Slots per expert of one tile.
__global__ __launch_bounds__(256) void group_hist_kernel(GroupParams P) {
    extern __shared__ int32_t hist[];
    const Tile t = tile_of(P, blockIdx.x);
    for (int e = threadIdx.x; e < P.Epr; e += 256) hist[e] = 0;
    __syncthreads();
    int32_t ex[kSlotsPerThread];
    load_experts(P, t, ex);
#pragma unroll
    for (int j = 0; j < kSlotsPerThread; ++j)
        if (ex[j] >= 0) atomicAdd(&hist[ex[j]], 1);
    __syncthreads();
    int32_t *out = P.hist + (int64_t)blockIdx.x * P.Epr;
    for (int e = threadIdx.x; e < P.Epr; e += 256) out[e] = hist[e];
}

// The large form's scans.  First, per (segment, expert): the tiles' counts
// become their exclusive prefix sums, and the total goes behind the counts.
__global__ __launch_bounds__(256) void group_scan_tiles_kernel(GroupParams P, int32_t segments, int32_t segTiles) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= (int64_t)segments * P.Epr) return;
    const int32_t s = (int32_t)(c / P.Epr), e = (int32_t)(c - (int64_t)s * P.Epr);
    int32_t *col = P.hist + (int64_t)s * segTiles * P.Epr + e;
    int32_t sum = 0;
    for (int32_t i = 0; i < segTiles; i += 8) {
        int32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = i + j < segTiles ? col[(int64_t)(i + j) * P.Epr] : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (i + j < segTiles) col[(int64_t)(i + j) * P.Epr] = sum;
            sum += v[j];
        }
    }
    P.hist[(int64_t)P.W * P.tilesPerWindow * P.Epr + c] = sum;
}

// Exclusive prefix sum of the block's values (256 threads); *total gets the sum.
__device__ __forceinline__ int32_t block_excl_scan(int32_t v, int32_t *total) {
    __shared__ int32_t sums[kWaves];
    const int32_t incl = wave_incl_scan(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) sums[threadIdx.x >> 6] = incl;
    __syncthreads();
    int32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < (int)(threadIdx.x >> 6)) before += sums[w];
        all += sums[w];
    }
    *total = all;
    return before + incl - v;
}

// Second, the groups' starts from their totals: one block.
__global__ __launch_bounds__(256) void group_scan_groups_kernel(GroupParams P, int32_t groups) {
    const int32_t *totals = P.hist + (int64_t)P.W * P.tilesPerWindow * P.Epr;
    int32_t carry = 0;
    for (int32_t g0 = 0; g0 < groups; g0 += 256) {
        const int32_t g = g0 + threadIdx.x;
        int32_t all;
        const int32_t at = block_excl_scan(g < groups ? totals[g] : 0, &all);
        if (g < groups) P.offsets[g] = carry + at;
        carry += all;
    }
    if (threadIdx.x == 0) P.offsets[groups] = carry;
}

// Where the counts of the other tiles come from (header of this file).
constexpr int kCountAll = 0, kSumCounts = 1, kScanned = 2;

// LDS: cnt [kWaves][Epr], then base [Epr], then total [Epr].
template <int FROM>
__global__ __launch_bounds__(256) void group_place_kernel(GroupParams P, int32_t segTiles, int32_t bits) {
    extern __shared__ int32_t lds[];
    int32_t *cnt = lds, *base = lds + kWaves * P.Epr, *tot = base + P.Epr;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Tile t = tile_of(P, blockIdx.x);
    // this wave's quarter of the tile's slots, 64 at a time; requested first of all
    constexpr int kChunks = kSlotsPerThread;
    const int32_t w0 = wave * (kChunks * 64);
    int32_t ex[kChunks], rk[kChunks];
    float wt[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int32_t i = w0 + c * 64 + lane;
        ex[c] = i < t.slots ? P.expertIds[t.slot0 + i] : -1;
        wt[c] = P.weights && i < t.slots ? P.weights[t.slot0 + i] : 0.0f;
    }
    for (int e = threadIdx.x; e < (kWaves + 2) * P.Epr; e += 256) lds[e] = 0;
    __syncthreads();
    const int32_t groups0 = t.segment * P.Epr;
    if (FROM != kScanned) {
        int32_t before = 0;  // entries of the segments in front
        const int32_t mine = (blockIdx.x - t.segTile0) * P.Epr;
        if (FROM == kCountAll) {
            // all slots in order, up to the segment's end
            __shared__ int32_t live[64];  // slots of valid rows, per window
            if ((int)threadIdx.x < P.W)
                live[threadIdx.x] = P.K * (P.recvCount ? min(max(P.recvCount[threadIdx.x], 0), P.M) : P.M);
            __syncthreads();
            const int32_t slots = P.M * P.K, end = (P.rank < 0 ? t.window + 1 : P.W) * slots;
            for (int32_t i0 = 0; i0 < end; i0 += 256 * 16) {
                int32_t id[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int32_t i = i0 + j * 256 + threadIdx.x;
                    id[j] = i < end ? P.expertIds[i] : -1;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int32_t i = i0 + j * 256 + threadIdx.x;
                    const int32_t w = min((int32_t)div_by((uint32_t)i, P.windowDiv), P.W - 1);
                    const int32_t e = id[j] - (P.rank < 0 ? w : P.rank) * P.Epr;
                    if (i >= end || (uint32_t)e >= (uint32_t)P.Epr || i - w * slots >= live[w]) continue;
                    if (P.rank < 0 && w < t.segment) {
                        ++before;
                    } else {
                        atomicAdd(&tot[e], 1);
                        if (i < t.slot0) atomicAdd(&base[e], 1);
                    }
                }
            }
        } else {
            const int64_t seg0 = (int64_t)t.segTile0 * P.Epr;
            const int32_t words = segTiles * P.Epr;
            for (int64_t i0 = 0; i0 < seg0; i0 += 256 * 8) {
                int32_t v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int64_t i = i0 + j * 256 + threadIdx.x;
                    v[j] = i < seg0 ? P.hist[i] : 0;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) before += v[j];
            }
            for (int32_t i0 = 0; i0 < words; i0 += 256 * 8) {
                int32_t v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int32_t i = i0 + j * 256 + threadIdx.x;
                    v[j] = i < words ? P.hist[seg0 + i] : 0;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (v[j] == 0) continue;
                    const int32_t i = i0 + j * 256 + threadIdx.x, e = (int32_t)((uint32_t)i % (uint32_t)P.Epr);
                    atomicAdd(&tot[e], v[j]);
                    if (i < mine) atomicAdd(&base[e], v[j]);
                }
            }
        }
        __syncthreads();
        int32_t carry;
        block_excl_scan(before, &carry);
        for (int32_t e0 = 0; e0 < P.Epr; e0 += 256) {
            const int32_t e = e0 + threadIdx.x;
            int32_t all;
            const int32_t at = carry + block_excl_scan(e < P.Epr ? tot[e] : 0, &all);
            if (e < P.Epr) {
                base[e] += at;
                if (mine == 0) P.offsets[groups0 + e] = at;
            }
            carry += all;
        }
        if (threadIdx.x == 0 && mine == 0 && t.segTile0 + segTiles == (int32_t)gridDim.x) P.offsets[groups0 + P.Epr] = carry;
    } else {
        for (int e = threadIdx.x; e < P.Epr; e += 256)
            base[e] = P.offsets[groups0 + e] + P.hist[(int64_t)blockIdx.x * P.Epr + e];
    }
    __syncthreads();

    // Rank them, in order.
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        ex[c] -= t.firstExpert;
        if (w0 + c * 64 + lane >= t.live || (uint32_t)ex[c] >= (uint32_t)P.Epr) ex[c] = -1;
    }
    int32_t *mycnt = cnt + wave * P.Epr;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        uint64_t same = __ballot(ex[c] >= 0);
        for (int b = 0; b < bits; ++b) {
            const uint64_t one = __ballot((ex[c] >> b) & 1);
            same &= (ex[c] >> b) & 1 ? one : ~one;
        }
        const int32_t below = __popcll(same & ((1ull << lane) - 1ull));
        int32_t seen = 0;
        if (ex[c] >= 0) seen = mycnt[ex[c]];
        wave_lds_order();
        if (ex[c] >= 0 && below == 0) mycnt[ex[c]] = seen + __popcll(same);
        wave_lds_order();
        rk[c] = seen + below;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < P.Epr; e += 256) {  // counts -> bases of the waves
        int32_t at = base[e];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int32_t v = cnt[w * P.Epr + e];
            cnt[w * P.Epr + e] = at;
            at += v;
        }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int32_t i = w0 + c * 64 + lane;
        if (i >= t.slots) continue;
        const int64_t slot = t.slot0 + i;
        int32_t at = -1;
        if (ex[c] >= 0) {
            at = mycnt[ex[c]] + rk[c];
            P.entryRow[at] = (int32_t)(slot / P.K);
            if (P.weights) P.entryWeight[at] = wt[c];
        }
        P.entryOf[slot] = at;
    }
}

}  // namespace

int64_t group_scratch_words(int32_t W, int32_t M, int32_t K, int32_t Epr) {
    const int64_t tiles = (int64_t)W * group_tiles_per_window(M, K);
    return tiles * Epr + (int64_t)W * Epr;
}

hipError_t launch_group(const GroupParams &P, hipStream_t stream) {
    const int64_t tiles = (int64_t)P.W * P.tilesPerWindow;
    if (tiles > (1 << 23)) return hipErrorInvalidConfiguration;
    const int32_t segments = P.rank < 0 ? P.W : 1;
    const int32_t segTiles = (int32_t)(tiles / segments);
    const int64_t groups = (int64_t)segments * P.Epr;
    int32_t bits = 0;
    while ((1 << bits) < P.Epr) ++bits;
    const dim3 grid((uint32_t)tiles);
    const size_t lds = (size_t)(kWaves + 2) * P.Epr * sizeof(int32_t);
    if ((int64_t)P.W * P.M * P.K <= kGroupLocalSlots) {
        hipLaunchKernelGGL((group_place_kernel<kCountAll>), grid, dim3(256), lds, stream, P, segTiles, bits);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(group_hist_kernel, grid, dim3(256), P.Epr * sizeof(int32_t), stream, P);
    if (tiles * P.Epr <= kGroupSelfWords) {
        hipLaunchKernelGGL((group_place_kernel<kSumCounts>), grid, dim3(256), lds, stream, P, segTiles, bits);
    } else {
        hipLaunchKernelGGL(group_scan_tiles_kernel, dim3((uint32_t)ceil_div(groups, 256)), dim3(256), 0, stream, P, segments,
                           segTiles);
        hipLaunchKernelGGL(group_scan_groups_kernel, dim3(1), dim3(256), 0, stream, P, (int32_t)groups);
        hipLaunchKernelGGL((group_place_kernel<kScanned>), grid, dim3(256), lds, stream, P, segTiles, bits);
    }
    return hipGetLastError();
}

}  // namespace epdc
