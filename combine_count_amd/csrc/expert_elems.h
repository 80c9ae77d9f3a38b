// Elements of rows as the activation's and the int8 quantisation's kernels
// take them: eight at a time, bf16 or fp32 in memory, fp32 in registers.  Not
// part of the C ABI.
#pragma once

#include "tiles.h"

namespace epdc {
namespace {

struct Eight {
    float v[8];
};

// A grid's threads are counted in 32 bits: beyond this many blocks of 256 they go on to further rows.
constexpr int64_t kMostBlocks = 1 << 23;

// Eight elements on the way: 16 bytes of bf16, 32 of fp32.
template <bool FP32>
struct Raw8 {
    u32x4 w[FP32 ? 2 : 1];
};

template <bool FP32>
__device__ __forceinline__ Raw8<FP32> load_raw8(const uint8_t *row, int32_t unit) {  // elements 8 unit .. + 7
    const uint8_t *p = row + (int64_t)unit * (FP32 ? 32 : 16);
    Raw8<FP32> r;
#pragma unroll
    for (int i = 0; i < (FP32 ? 2 : 1); ++i) r.w[i] = load16<false>(p + i * 16);
    return r;
}

template <bool FP32>
__device__ __forceinline__ Eight to_eight(const Raw8<FP32> &r) {
    Eight e;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (FP32)
            e.v[i] = __uint_as_float(r.w[i / 4][i % 4]);
        else
            e.v[i] = __uint_as_float(i % 2 ? r.w[0][i / 2] & 0xffff0000u : r.w[0][i / 2] << 16);
    }
    return e;
}

template <bool FP32>
__device__ __forceinline__ void store_eight(uint8_t *row, int32_t unit, const Eight &e) {
    uint8_t *p = row + (int64_t)unit * (FP32 ? 32 : 16);
    if constexpr (FP32) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            store16<false>(p + i * 16, u32x4{__float_as_uint(e.v[4 * i]), __float_as_uint(e.v[4 * i + 1]),
                                             __float_as_uint(e.v[4 * i + 2]), __float_as_uint(e.v[4 * i + 3])});
    } else {
        store16<false>(p, u32x4{bf16_pair(e.v[0], e.v[1]), bf16_pair(e.v[2], e.v[3]), bf16_pair(e.v[4], e.v[5]),
                                bf16_pair(e.v[6], e.v[7])});
    }
}

// s(g) and 1 - s(g), neither by a difference: with t = exp(-|g|) <= 1 they are
// 1 / (1 + t) and t / (1 + t), the larger one s where g >= 0.
struct Sigmoid {
    float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid_of(float g) {
    const float t = expf(-fabsf(g)), large = 1.0f / (1.0f + t), small = t * large;
    return g >= 0.0f ? Sigmoid{large, small} : Sigmoid{small, large};
}

// The rows [first, last) that a call of `E` groups covers.
struct RowRange {
    int32_t first, last;
};
__device__ __forceinline__ RowRange rows_of_groups(const int32_t *offsets, int32_t E, int32_t maxEntries) {
    if (!offsets) return RowRange{0, maxEntries};
    return RowRange{min(max(offsets[0], 0), maxEntries), min(max(offsets[E], 0), maxEntries)};
}

// A row's place: a team of TEAM lanes (a wave, or a block of four) takes a row.
// Sum and maximum over the team, the same value in every lane; the sum's order
// is fixed.  `part` is the block's, one word a wave.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float *part) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    if constexpr (TEAM > 64) {
        __syncthreads();  // what the block read from `part` before
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = (part[0] + part[1]) + (part[2] + part[3]);
    }
    return v;
}
template <int TEAM>
__device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t *part) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
    if constexpr (TEAM > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = max(max(part[0], part[1]), max(part[2], part[3]));
    }
    return v;
}

}  // namespace
}  // namespace epdc
