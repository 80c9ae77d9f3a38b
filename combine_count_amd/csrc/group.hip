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
// Bases come from sums, not from atomics, so the order is fixed.  With more
// than kGroupSelfWords words of counts the sums of step 2 would read too much
// in every block: two scan launches between them turn the counts into bases.
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

// Slots per expert of one tile.
__global__ __launch_bounds__(256) void group_hist_kernel(GroupParams P) {
    extern __shared__ int32_t hist[];
    const Tile t = tile_of(P, blockIdx.x);
    for (int e = threadIdx.x; e < P.Epr; e += 256) hist[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < t.live; i += 256) {
        const int32_t e = P.expertIds[t.slot0 + i] - t.firstExpert;
        if ((uint32_t)e < (uint32_t)P.Epr) atomicAdd(&hist[e], 1);
    }
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

// SELF: the block sums the tiles' counts itself; else the scan launches left
// the bases.  LDS: cnt [kWaves][Epr], then base [Epr], then total [Epr].
template <bool SELF>
__global__ __launch_bounds__(256) void group_place_kernel(GroupParams P, int32_t segTiles, int32_t bits) {
    extern __shared__ int32_t lds[];
    int32_t *cnt = lds, *base = lds + kWaves * P.Epr, *tot = base + P.Epr;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Tile t = tile_of(P, blockIdx.x);
    for (int e = threadIdx.x; e < (kWaves + 2) * P.Epr; e += 256) lds[e] = 0;
    __syncthreads();
    const int32_t groups0 = t.segment * P.Epr;
    if (SELF) {
        int32_t before = 0;  // entries of the segments in front
        const int64_t seg0 = (int64_t)t.segTile0 * P.Epr;
        for (int64_t i = threadIdx.x; i < seg0; i += 256) before += P.hist[i];
        const int32_t words = segTiles * P.Epr, mine = (blockIdx.x - t.segTile0) * P.Epr;
        for (int32_t i = threadIdx.x; i < words; i += 256) {
            const int32_t v = P.hist[seg0 + i];
            if (v == 0) continue;
            const int32_t e = i % P.Epr;
            atomicAdd(&tot[e], v);
            if (i < mine) atomicAdd(&base[e], v);
        }
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

    // Rank the wave's quarter of the slots, in order.
    constexpr int kChunks = kGroupTileSlots / (64 * kWaves);  // 64-slot chunks per wave
    const int32_t w0 = wave * (kChunks * 64);
    int32_t ex[kChunks], rk[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int32_t i = w0 + c * 64 + lane;
        int32_t e = -1;
        if (i < t.live) {
            e = P.expertIds[t.slot0 + i] - t.firstExpert;
            if ((uint32_t)e >= (uint32_t)P.Epr) e = -1;
        }
        ex[c] = e;
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
            if (P.weights) P.entryWeight[at] = P.weights[slot];
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
    hipLaunchKernelGGL(group_hist_kernel, grid, dim3(256), P.Epr * sizeof(int32_t), stream, P);
    if (tiles * P.Epr <= kGroupSelfWords) {
        hipLaunchKernelGGL((group_place_kernel<true>), grid, dim3(256), lds, stream, P, segTiles, bits);
    } else {
        hipLaunchKernelGGL(group_scan_tiles_kernel, dim3((uint32_t)ceil_div(groups, 256)), dim3(256), 0, stream, P, segments,
                           segTiles);
        hipLaunchKernelGGL(group_scan_groups_kernel, dim3(1), dim3(256), 0, stream, P, (int32_t)groups);
        hipLaunchKernelGGL((group_place_kernel<false>), grid, dim3(256), lds, stream, P, segTiles, bits);
    }
    return hipGetLastError();
}

}  // namespace epdc
