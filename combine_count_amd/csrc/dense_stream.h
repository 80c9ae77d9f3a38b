// The product of bf16 or int8 rows where there are few of them: the weights are
// streamed once, at the rate of the memory, by enough blocks to ask for them.
//
// v_mfma_f32_16x16x32_bf16 (v_mfma_i32_16x16x64_i8): lane l holds row (or
// column) l % 16, bytes [16 (l/16), 16 (l/16) + 16) of 64 of the summed index;
// of the result column l % 16, rows 4 (l/16) .. + 3.  The weights are the
// instruction's rows.
//
// A block takes 16 FN columns and 16 FM entries of one expert; its four waves
// share the row's bytes out among them (128-byte chunks in turn) and add their
// sums up at the end, in LDS, in wave order.  No wave needs another's operands,
// so they go straight from memory into registers, DEPTH chunks ahead, with no
// barrier on the way.  7168 -> 4096, bf16: one expert, 16 entries 28 us (2.1 TB/s:
// 128 blocks, half the CUs), 4 experts, 16 entries 49 us (4.8 TB/s); int8 16 and
// 26 us.
#pragma once

#include "tiles.h"

namespace epdc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ i32x4 mfma16(u32x4 a, u32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

template <bool INT8, int FM, int FN, int DEPTH, bool OUT32>
__global__ __launch_bounds__(256) void dense_stream_kernel(DenseParams P) {
    using Sum4 = std::conditional_t<INT8, i32x4, f32x4>;
    using Sum = std::conditional_t<INT8, int32_t, float>;
    constexpr int BM = 16 * FM, BN = 16 * FN;
    __shared__ __attribute__((aligned(16))) Sum part[4][BM][BN + 4];  // + 4: rows on other banks
    __shared__ int32_t rows[BM];
    const int32_t NT = ceil_div(P.N, BN), rowBytes = P.H * (INT8 ? 1 : 2);
    Groups groups = count_tiles<BM>(P, NT);
    const TileAt T = find_tile<BM, BN>(P, groups, NT, blockIdx.x);
    if (T.e < 0) return;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int r16 = lane & 15, kb = lane >> 4;
    const uint8_t *m[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        const int32_t ent = min(T.m0 + f * 16 + r16, T.hi - 1);
        const int32_t r = P.entryRow ? P.entryRow[ent] : ent;
        const bool in = (uint32_t)r < (uint32_t)P.numRows;
        if (wave == 0 && kb == 0) rows[f * 16 + r16] = in ? r : -1;
        m[f] = P.rows + (int64_t)(in ? r : 0) * rowBytes + kb * 16;
    }
    uint32_t n[FN];
    const uint8_t *const first = P.weights + ((int64_t)T.e * P.N + T.n0) * rowBytes;
#pragma unroll
    for (int f = 0; f < FN; ++f) n[f] = (uint32_t)min(f * 16 + r16, P.N - 1 - T.n0) * (uint32_t)rowBytes + kb * 16;
    struct Chunk {
        u32x4 m[FM][2], n[FN][2];
    };
    auto load = [&](Chunk &c, int at) {  // chunk `at`, whole
        const int64_t k = (int64_t)uniform(at) * 128;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            c.n[f][0] = load16<true>(first + k + n[f]);
            c.n[f][1] = load16<true>(first + k + 64 + n[f]);
        }
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            c.m[f][0] = load16<false>(m[f] + k);
            c.m[f][1] = load16<false>(m[f] + k + 64);
        }
    };
    auto load_tail = [&](Chunk &c, int at) {  // the last chunk, which the rows end in: zeros behind their end, on both sides
        const int64_t k = (int64_t)at * 128;
        const u32x4 none = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool in = k + h * 64 + kb * 16 < rowBytes;
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                const u32x4 v = load16<false>(first + n[f] + (in ? k + h * 64 : -kb * 16));
                c.n[f][h] = in ? v : none;
            }
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const u32x4 v = load16<false>(m[f] + (in ? k + h * 64 : -kb * 16));
                c.m[f][h] = in ? v : none;
            }
        }
    };
    Sum4 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = Sum4{0, 0, 0, 0};
    auto multiply = [&](const Chunk &c) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) acc[i][j] = mfma16(c.n[i][h], c.m[j][h], acc[i][j]);
    };
    const int whole = rowBytes / 128;                            // whole chunks
    const int mine = whole > wave ? (whole - wave + 3) / 4 : 0;  // chunks wave, wave + 4, ...
    Chunk c[DEPTH];
    if (mine > 0) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load(c[d], wave + 4 * min(d, mine - 1));
        int i = 0;
        for (; i + 2 * DEPTH <= mine; i += DEPTH) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                multiply(c[d]);
                load(c[d], wave + 4 * (i + DEPTH + d));
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (i + d < mine) {
                multiply(c[d]);
                if (i + DEPTH + d < mine) load(c[d], wave + 4 * (i + DEPTH + d));
            }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (i + DEPTH + d < mine) multiply(c[d]);
    }
    if (rowBytes % 128 != 0 && (whole & 3) == wave) {
        load_tail(c[0], whole);
        multiply(c[0]);
    }
    // lane: entry r16 of fragment j, columns 4 kb .. + 3 of fragment i
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) *reinterpret_cast<Sum4 *>(&part[wave][j * 16 + r16][i * 16 + kb * 4]) = acc[i][j];
    __syncthreads();
    constexpr int kPer = OUT32 ? 4 : 8;  // columns per thread: 16 bytes of results
    for (int u = threadIdx.x; u < BM * BN / kPer; u += 256) {
        const int ent = u / (BN / kPer), col = (u - ent * (BN / kPer)) * kPer;
        if (T.m0 + ent >= T.hi || T.n0 + col >= P.N) continue;
        float v[kPer];
        const int32_t row = rows[ent];  // -1: a row of zeros
        const float w = P.entryWeight ? P.entryWeight[T.m0 + ent] : 1.0f;
        float scale = 1.0f;
        if constexpr (INT8) scale = row < 0 ? 0.0f : P.rowScales[row];
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const Sum sum = ((part[0][ent][col + q] + part[1][ent][col + q]) + part[2][ent][col + q]) + part[3][ent][col + q];
            v[q] = (float)sum;
            if constexpr (INT8) v[q] = v[q] * scale * P.weightScales[(int64_t)T.e * P.N + T.n0 + col + q];
            v[q] = row < 0 ? 0.0f : v[q] * w;
        }
        const int64_t o = (int64_t)(T.m0 + ent) * P.N + T.n0 + col;
        if constexpr (OUT32)
            *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(P.out) + o) = f32x4{v[0], v[1], v[2], v[3]};
        else
            *reinterpret_cast<u32x4 *>(reinterpret_cast<uint16_t *>(P.out) + o) =
                u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
    }
}

template <bool INT8, int FM, int FN, int DEPTH>
hipError_t launch_stream(const DenseParams &P, bool out32, hipStream_t stream) {
    const int64_t tiles = ((int64_t)P.maxEntries / (16 * FM) + (P.E < P.maxEntries ? P.E : P.maxEntries)) * ceil_div(P.N, 16 * FN);
    const int64_t blocks = (tiles + 7) / 8 * 8;
    if (blocks > (1 << 23)) return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)blocks);
    if (out32)
        hipLaunchKernelGGL((dense_stream_kernel<INT8, FM, FN, DEPTH, true>), grid, dim3(256), 0, stream, P);
    else
        hipLaunchKernelGGL((dense_stream_kernel<INT8, FM, FN, DEPTH, false>), grid, dim3(256), 0, stream, P);
    return hipGetLastError();
}

}  // namespace
}  // namespace epdc
