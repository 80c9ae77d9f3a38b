// The products of bf16 and int8 rows with the experts' weights, and the bf16
// product's two gradients, for gfx950: over a group's entries i
//   product           out[i][n]   = sum_h rows[r_i][h] W[n][h]
//   rows' gradient    dRows[i][h] = sum_n dOut[r_i][n] W[n][h]
//   weights' gradient dW[n][h]    = sum_i dOut[o_i][n] rows[r_i][h]
//
// One form for all: 64 x 64 tiles, both operands brought into LDS with the
// summed index running along a row, 32 x 32 of the tile per wave with
// v_mfma_f32_32x32x16_bf16 (v_mfma_i32_32x32x32_i8).
#include "tiles.h"

namespace epdc {
namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <DenseKind KIND, bool INT8, bool OUT32>
__global__ __launch_bounds__(256) void dense_kernel(DenseParams P) {
    using Acc = std::conditional_t<INT8, i32x16, f32x16>;
    using Elem = std::conditional_t<INT8, uint8_t, uint16_t>;
    constexpr int kStep = INT8 ? 64 : 32;  // elements of the summed index a step
    __shared__ __attribute__((aligned(16))) uint8_t left[64][80], right[64][80];
    __shared__ int32_t rowOf[64], outOf[64];
    const int32_t C = KIND == kDenseProduct ? P.N : P.H;  // columns of the output
    TileAt T;
    int32_t r0 = 0;  // weights' gradient: first row of the tile
    if constexpr (KIND == kDenseWeightsGrad) {
        const int32_t RT = ceil_div(P.N, 64), CT = ceil_div(P.H, 64);
        const int64_t at = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
        if (at >= (int64_t)P.E * RT * CT) return;
        const int32_t e = (int32_t)(at / (RT * CT)), rest = (int32_t)(at - (int64_t)e * RT * CT);
        Groups g;
        int32_t least = P.maxEntries;
        for (int32_t e0 = (P.E - 1) & ~63; e0 >= (e & ~63); e0 -= 64) load_groups<64>(P, e0, least, g);
        T = TileAt{e, uniform(__shfl(g.lo, e & 63)), uniform(__shfl(g.hi, e & 63)), rest % CT * 64};
        r0 = rest / CT * 64;
    } else {
        const int32_t NT = ceil_div(C, 64);
        Groups g = count_tiles<64>(P, NT);
        T = find_tile<64, 64>(P, g, NT, blockIdx.x);
        if (T.e < 0) return;
        if (threadIdx.x < 64) {
            const int32_t ent = T.m0 + threadIdx.x;
            const int32_t r = ent < T.hi ? (P.entryRow ? P.entryRow[ent] : ent) : -1;
            rowOf[threadIdx.x] = (uint32_t)r < (uint32_t)P.numRows ? r : -1;
        }
    }
    const int32_t K = KIND == kDenseProduct ? P.H : KIND == kDenseRowsGrad ? P.N : T.hi - T.m0;
    const Elem *rows = reinterpret_cast<const Elem *>(P.rows), *dOut = reinterpret_cast<const Elem *>(P.dOut);
    const Elem *w = reinterpret_cast<const Elem *>(P.weights) + (int64_t)T.e * P.N * P.H;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wr = (wave & 1) * 32, wc = (wave >> 1) * 32;
    Acc acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0;
    for (int32_t k0 = 0; k0 < K; k0 += kStep) {
        __syncthreads();
        if constexpr (KIND == kDenseWeightsGrad) {
            if (threadIdx.x < kStep) {
                const int32_t ent = T.m0 + k0 + threadIdx.x;
                int32_t r = -1, o = -1;
                if (ent < T.hi) {
                    r = P.entryRow ? P.entryRow[ent] : ent;
                    o = P.outRow ? P.outRow[ent] : ent;
                    if ((uint32_t)r >= (uint32_t)P.numRows || (uint32_t)o >= (uint32_t)P.numOutRows) r = o = -1;
                }
                rowOf[threadIdx.x] = r;
                outOf[threadIdx.x] = o;
            }
            __syncthreads();
        }
        for (int u = threadIdx.x; u < 64 * kStep; u += 256) {
            const int x = KIND == kDenseProduct ? u / kStep : u % 64, kk = KIND == kDenseProduct ? u % kStep : u / 64;
            const int32_t k = k0 + kk, c = T.n0 + x;
            Elem a = 0, b = 0;  // of the output's columns, of its rows
            if constexpr (KIND == kDenseProduct) {
                if (k < K && c < C) a = w[(int64_t)c * P.H + k];
                if (k < K && rowOf[x] >= 0) b = rows[(int64_t)rowOf[x] * P.H + k];
            } else if constexpr (KIND == kDenseRowsGrad) {
                if (k < K && c < C) a = w[(int64_t)k * P.H + c];
                if (k < K && rowOf[x] >= 0) b = rows[(int64_t)rowOf[x] * P.N + k];
            } else {
                if (k < K && rowOf[kk] >= 0) {
                    if (c < C) a = rows[(int64_t)rowOf[kk] * P.H + c];
                    if (r0 + x < P.N) b = dOut[(int64_t)outOf[kk] * P.N + r0 + x];
                }
            }
            reinterpret_cast<Elem *>(left[x])[kk] = a;
            reinterpret_cast<Elem *>(right[x])[kk] = b;
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const u32x4 a = *reinterpret_cast<const u32x4 *>(&left[wc + (lane & 31)][s * 32 + (lane >> 5) * 16]);
            const u32x4 b = *reinterpret_cast<const u32x4 *>(&right[wr + (lane & 31)][s * 32 + (lane >> 5) * 16]);
            if constexpr (INT8)
                acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), acc, 0, 0, 0);
            else
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
        }
    }
    // lane: row l % 32 of the output, columns 8 (i / 4) + 4 (l / 32) + i % 4
    const int32_t m = wr + (lane & 31);
    int64_t row;
    bool in, none = false;
    float wgt = 1.0f;
    if constexpr (KIND == kDenseWeightsGrad) {
        row = (int64_t)T.e * P.N + r0 + m;
        in = r0 + m < P.N;
    } else {
        row = T.m0 + m;
        in = T.m0 + m < T.hi;
        if (in) none = rowOf[m] < 0;
        if (in && P.entryWeight) wgt = P.entryWeight[row];
    }
    if (!in) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int32_t c = T.n0 + wc + 8 * (i / 4) + 4 * (lane >> 5) + i % 4;
        if (c >= C) continue;
        float v;
        if constexpr (INT8)
            v = none ? 0.0f : (float)acc[i] * P.rowScales[rowOf[m]] * P.weightScales[(int64_t)T.e * P.N + c];
        else
            v = acc[i];
        v = none ? 0.0f : v * wgt;
        const int64_t o = row * C + c;
        if (KIND == kDenseWeightsGrad && P.base)
            v += OUT32 ? reinterpret_cast<const float *>(P.base)[o] : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(P.base)[o] << 16);
        if (OUT32)
            reinterpret_cast<float *>(P.out)[o] = v;
        else
            reinterpret_cast<uint16_t *>(P.out)[o] = (uint16_t)bf16_rne(v);
    }
}

template <DenseKind KIND, bool INT8>
hipError_t launch_kind(const DenseParams &P, bool out32, hipStream_t stream) {
    dim3 grid;
    if (KIND == kDenseWeightsGrad) {
        const int64_t tiles = (int64_t)P.E * ceil_div(P.N, 64) * ceil_div(P.H, 64);
        if (tiles > ((int64_t)1 << 38)) return hipErrorInvalidConfiguration;
        grid = tiles < (1 << 22) ? dim3((uint32_t)tiles) : dim3(1 << 22, (uint32_t)((tiles + (1 << 22) - 1) >> 22));
    } else {
        const int64_t tiles = ((int64_t)P.maxEntries / 64 + (P.E < P.maxEntries ? P.E : P.maxEntries)) * ceil_div(KIND == kDenseProduct ? P.N : P.H, 64);
        if (tiles > (1 << 23)) return hipErrorInvalidConfiguration;
        grid = dim3((uint32_t)((tiles + 7) / 8 * 8));
    }
    if (out32)
        hipLaunchKernelGGL((dense_kernel<KIND, INT8, true>), grid, dim3(256), 0, stream, P);
    else
        hipLaunchKernelGGL((dense_kernel<KIND, INT8, false>), grid, dim3(256), 0, stream, P);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dense(const DenseParams &P, DenseKind kind, bool int8, bool out32, hipStream_t stream) {
    if (int8) return launch_kind<kDenseProduct, true>(P, out32, stream);
    if (kind == kDenseProduct) return launch_kind<kDenseProduct, false>(P, out32, stream);
    if (kind == kDenseRowsGrad) return launch_kind<kDenseRowsGrad, false>(P, out32, stream);
    return launch_kind<kDenseWeightsGrad, false>(P, out32, stream);
}

}  // namespace epdc
