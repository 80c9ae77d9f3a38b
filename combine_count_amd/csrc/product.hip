// The experts' product for gfx950: out[i] = w_i * rows[r_i] . weights[e]^T for
// every entry i of every expert e, fp4x2 rows and weights with block scales.
//
// v_mfma_scale_f32_16x16x128_f8f6f4: D[16][16] += A[16][128] B[128][16], each
// operand element times its 32-block's power-of-two scale, fp32 sums.  Lane l
// holds row (or column) l % 16, elements [32 (l/16), 32 (l/16) + 32) -- one
// block, 16 bytes -- and that block's scale byte; of the result column l % 16,
// rows 4 (l/16) .. + 3.
#include "ops_internal.h"

namespace epdc {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;  // the instruction's operand format

__device__ __forceinline__ f32x4 mfma_fp4(u32x4 a, u32x4 b, f32x4 c, int32_t sa, int32_t sb) {
    const i32x8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const i32x8 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, kFp4, kFp4, 0, sa, 0, sb);
}

// Entries of expert e, both ends inside [0, maxEntries].
__device__ __forceinline__ void group_range(const ProductParams &P, int32_t e, int32_t &lo, int32_t &hi) {
    lo = min(max(P.offsets[e], 0), P.maxEntries);
    hi = min(max(P.offsets[e + 1], lo), P.maxEntries);
}

// One wave per 16 columns and 32 rows of one expert; grid (column tiles, row
// tiles, experts).  Operands straight from memory.
template <bool OUT32>
__global__ __launch_bounds__(256) void product_simple_kernel(ProductParams P) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int32_t e = blockIdx.z;
    int32_t lo, hi;
    group_range(P, e, lo, hi);
    const int32_t n0 = (blockIdx.x * 4 + wave) * 16;
    if (n0 >= P.N) return;
    const int32_t col = n0 + (lane & 15);
    const bool colIn = col < P.N;
    const uint8_t *b = P.weights + ((int64_t)e * P.N + (colIn ? col : 0)) * P.rowBytes;
    const uint8_t *bs = P.weightScales + ((int64_t)e * P.N + (colIn ? col : 0)) * P.words * 4;
    for (int32_t m0 = lo + blockIdx.y * 32; m0 < hi; m0 += gridDim.y * 32) {
        const uint8_t *a[2], *as[2];
        bool in[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int32_t ent = m0 + i * 16 + (lane & 15);
            int32_t r = -1;
            if (ent < hi) r = P.entryRow ? P.entryRow[ent] : ent;
            in[i] = r >= 0 && r < P.numRows;
            a[i] = P.rows + (int64_t)(in[i] ? r : 0) * P.rowBytes;
            as[i] = P.rowScales + (int64_t)(in[i] ? r : 0) * P.words * 4;
        }
        f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        for (int32_t k = 0; k < P.rowBytes; k += 64) {
            const int32_t at = k + (lane >> 4) * 16;
            const bool kin = at < P.rowBytes;
            u32x4 bv = {0, 0, 0, 0};
            int32_t sb = 127;
            if (kin && colIn) bv = load16<false>(b + at), sb = bs[at >> 4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                u32x4 av = {0, 0, 0, 0};
                int32_t sa = 127;
                if (kin && in[i]) av = load16<false>(a[i] + at), sa = as[i][at >> 4];
                acc[i] = mfma_fp4(av, bv, acc[i], sa, sb);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t ent = m0 + i * 16 + (lane >> 4) * 4 + j;
                if (ent >= hi || !colIn) continue;
                float v = acc[i][j];
                if (P.entryWeight) v *= P.entryWeight[ent];
                const int64_t o = (int64_t)ent * P.N + col;
                if (OUT32)
                    static_cast<float *>(P.out)[o] = v;
                else
                    static_cast<uint16_t *>(P.out)[o] = (uint16_t)bf16_rne(v);
            }
    }
}

}  // namespace

hipError_t launch_product(const ProductParams &P, bool out32, hipStream_t stream) {
    if (P.maxEntries == 0) return hipSuccess;
    const int32_t per = ceil_div(P.maxEntries, 32 * P.E);
    const dim3 grid((uint32_t)ceil_div(P.N, 64), (uint32_t)(per < 1024 ? per : 1024), (uint32_t)P.E);
    if (out32)
        hipLaunchKernelGGL((product_simple_kernel<true>), grid, dim3(256), 0, stream, P);
    else
        hipLaunchKernelGGL((product_simple_kernel<false>), grid, dim3(256), 0, stream, P);
    return hipGetLastError();
}

}  // namespace epdc
