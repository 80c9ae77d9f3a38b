// What the products' kernels share (product.hip, product_dense.h): vector
// types, loads straight into LDS, and which tile of which expert a block
// takes.  Not part of the C ABI.
#pragma once

#include "ops_internal.h"

namespace epdc {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Behind inline matrix instructions, before their sums are read.
__device__ __forceinline__ void mfma_done() { asm volatile("s_nop 15\n\ts_nop 15"); }

// Two values as bf16, the first low, rounded to nearest even.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// 16 bytes per lane from memory into LDS at lds + lane * 16 (lds the same in
// all lanes), counted by vmcnt: from rs' base at voff (per lane) + soff.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t rs, uint32_t voff, int32_t soff, uint8_t *lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void *)lds, 16, (int)voff, soff, 0, 0);
}
__device__ __forceinline__ void load_lds16(const uint8_t *src, uint8_t *lds) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                     (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t *base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, 0xffffffff, 0x00020000);
}

// Where a block's tile lies: expert, entries [m0, hi), columns from n0.
struct TileAt {
    int32_t e, m0, hi, n0;
};

// The groups as a wave holds them, 64 experts at a time (experts e0 + lane):
// entries [lo, hi) and the row tiles up to and with the lane's expert.  The
// experts are gone through from the last to the first: a group ends at the
// smallest offset behind its start's, so that groups never share an entry,
// whatever the offsets are.
struct Groups {
    int32_t lo, hi, incl;
    int64_t total;  // tiles of all experts
};

// Loads the groups of experts e0 ..; `least` is the smallest offset behind
// them (maxEntries at first) and becomes that behind e0 - 1's start.
template <int BM, class Params>
__device__ __forceinline__ void load_groups(const Params &P, int32_t e0, int32_t &least, Groups &g) {
    const int lane = threadIdx.x & 63, e = e0 + lane;
    int32_t end = e < P.E ? min(max(P.offsets[e + 1], 0), P.maxEntries) : P.maxEntries;
    g.lo = e < P.E ? min(max(P.offsets[e], 0), P.maxEntries) : P.maxEntries;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_down(end, d);
        if (lane + d < 64) end = min(end, o);
    }
    end = min(end, least);
    g.hi = e < P.E ? max(end, g.lo) : g.lo;
    g.incl = wave_incl_scan((g.hi - g.lo + BM - 1) / BM);
    least = uniform(min(end, g.lo));  // of lane 0
}

template <int BM, class Params>
__device__ __forceinline__ Groups count_tiles(const Params &P, int32_t NT) {
    Groups g;
    int64_t total = 0;
    int32_t least = P.maxEntries;
    for (int32_t e0 = (P.E - 1) & ~63; e0 >= 0; e0 -= 64) {
        load_groups<BM>(P, e0, least, g);
        total += uniform(__shfl(g.incl, 63));
    }
    g.total = total * NT;
    return g;
}

// A tile among its expert's: group [lo, hi), row tile m of `tiles`, columns from n0.
struct PlaceOf {
    int32_t e, lo, hi, m, tiles, n0;
};

// Tile b among all experts' tiles (BM entries x BN columns), or e = -1 when
// there are fewer.  Each XCD (block b % 8) takes a contiguous stretch of the
// tiles, so the tiles that run on it together share operands in its L2;
// within an expert, bands of four row tiles (up to seven where four would
// leave a rest) go through the columns together.
template <int BM, int BN, class Params>
__device__ __forceinline__ PlaceOf find_place(const Params &P, Groups &g, int32_t NT, int32_t b) {
    const int64_t per = (g.total + 7) / 8;
    const int64_t at = (b & 7) * per + (b >> 3);
    PlaceOf t{-1, 0, 0, 0, 0, 0};
    if ((b >> 3) >= per || at >= g.total) return t;
    int64_t before = 0;
    int32_t least = P.maxEntries;
    for (int32_t e0 = (P.E - 1) & ~63; e0 >= 0; e0 -= 64) {
        if (P.E > 64) load_groups<BM>(P, e0, least, g);
        const uint64_t past = __ballot((before + g.incl) * NT > at);
        if (past) {
            const int f = __builtin_ctzll(past);
            const int32_t lo = __builtin_amdgcn_readlane(g.lo, f), hi = __builtin_amdgcn_readlane(g.hi, f);
            const int32_t tiles = (hi - lo + BM - 1) / BM;
            const int32_t r0 = (int32_t)(at - (before + __builtin_amdgcn_readlane(g.incl, f) - tiles) * NT);  // inside the expert
            const int32_t size = ceil_div(tiles, max(tiles >> 2, 1));  // row tiles of a band
            const int32_t band = r0 / (size * NT), rows = min(size, tiles - band * size), r = r0 - band * size * NT;
            const int32_t n = r / rows, m = band * size + r - n * rows;
            return PlaceOf{e0 + f, lo, hi, m, tiles, n * BN};
        }
        before += uniform(__shfl(g.incl, 63));
    }
    return t;
}

template <int BM, int BN, class Params>
__device__ __forceinline__ TileAt find_tile(const Params &P, Groups &g, int32_t NT, int32_t b) {
    const PlaceOf t = find_place<BM, BN>(P, g, NT, b);
    if (t.e < 0) return TileAt{-1, 0, 0, 0};
    return TileAt{uniform(t.e), uniform(t.lo + t.m * BM), uniform(min(t.hi, t.lo + t.m * BM + BM)), uniform(t.n0)};
}

}  // namespace
}  // namespace epdc
