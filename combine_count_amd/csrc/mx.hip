// fp4x2 rows with block scales (OCP microscaling, MXFP4) for gfx950.
//
// quantise:    per 32-element block, m = the largest magnitude, scale byte
//              b = clamp(floor(log2 m) - 2 + 127, 0, 254): 2 is the exponent
//              of e2m1's largest value (6 = 1.5 * 2^2), so the block's largest
//              element lands in [4, 8) and saturates at 6; codes by the
//              hardware's scaled conversion, nearest even.
// dequantise:  code value * 2^(b - 127) by the hardware's scaled conversion.
//
// Both are bound by memory: a thread's share is 8 elements (16 bytes of bf16,
// 32 of fp32, 4 bytes of codes), four such units in flight; a block of 32 is
// four lanes, so its maximum takes two exchanges inside a group of four lanes.
// 16384 x 7168 bf16: quantise 52 us (5.7 TB/s), dequantise of the same codes
// 43 us (6.9, part of them out of the memory-side cache); 128 rows 3.5 and 3.1.
#include "ops_internal.h"

namespace epdc {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kUnits = 4;  // units of 8 elements in flight per thread

// Units of a block of threads: `first` + j * 256 + threadIdx.x.  Splits the
// unit into its row and place once per block in 64 bits, then in 32.
struct Place {
    int64_t row;
    uint32_t at;  // unit in its row
    bool live;
};

__device__ __forceinline__ Place place_of(const MxParams &P, int64_t blockRow, uint32_t blockAt, int64_t unit, uint32_t step) {
    const uint32_t n = blockAt + step;
    const uint32_t r = div_by(n, P.rowDiv);
    Place pl;
    pl.row = blockRow + r;
    pl.at = n - r * (uint32_t)P.unitsPerRow;
    pl.live = unit < P.units;
    if (pl.live && P.rowCount) {
        const uint32_t w = div_by((uint32_t)pl.row, P.winDiv);
        pl.live = (int32_t)((uint32_t)pl.row - w * (uint32_t)P.M) < P.rowCount[w];
    }
    return pl;
}

// Largest value of a 32-bit word over each group of four lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));  // lanes 1 0 3 2
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));  // lanes 2 3 0 1
}

template <bool FP32>
__global__ __launch_bounds__(256) void mx_quantize_kernel(MxParams P) {
    const int64_t first = (int64_t)blockIdx.x * (256 * kUnits);
    const int64_t blockRow = first / P.unitsPerRow;
    const uint32_t blockAt = (uint32_t)(first - blockRow * P.unitsPerRow);
    Place pl[kUnits];
    u32x4 v[kUnits][FP32 ? 2 : 1];
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
        const uint32_t step = j * 256 + threadIdx.x;
        const int64_t unit = first + step;
        pl[j] = place_of(P, blockRow, blockAt, unit, step);
        const uint8_t *src = P.in + unit * (FP32 ? 32 : 16);
        v[j][0] = u32x4{0, 0, 0, 0};
        if (FP32) v[j][1] = u32x4{0, 0, 0, 0};
        if (pl[j].live) {
            v[j][0] = load16<true>(src);
            if (FP32) v[j][1] = load16<true>(src + 16);
        }
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
        // the largest magnitude's bits: an infinity or a NaN is the largest of all
        uint32_t m = 0;
        if (FP32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, v[j][i >> 2][i & 3] & 0x7fffffffu);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m = max(m, v[j][0][i] & 0x7fff0000u);
                m = max(m, (v[j][0][i] << 16) & 0x7fff0000u);
            }
        }
        m = quad_max(m);
        const uint32_t exponent = m >> 23;
        const uint32_t byte = exponent == 255 ? 255 : exponent < 2 ? 0 : exponent - 2;
        const float scale = __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);  // 2^-127 is subnormal
        uint32_t codes = 0;
        if (FP32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float a = __uint_as_float(v[j][i][0]), b = __uint_as_float(v[j][i][1]);
                const float c = __uint_as_float(v[j][i][2]), d = __uint_as_float(v[j][i][3]);
                if (i == 0) {
                    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, a, b, scale, 0);
                    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, c, d, scale, 1);
                } else {
                    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, a, b, scale, 2);
                    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, c, d, scale, 3);
                }
            }
        } else {
            // (a bit cast of a vector's element would take its first: copies)
            const uint32_t w0 = v[j][0].x, w1 = v[j][0].y, w2 = v[j][0].z, w3 = v[j][0].w;
            codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, __builtin_bit_cast(bf16x2, w0), scale, 0);
            codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, __builtin_bit_cast(bf16x2, w1), scale, 1);
            codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, __builtin_bit_cast(bf16x2, w2), scale, 2);
            codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, __builtin_bit_cast(bf16x2, w3), scale, 3);
        }
        if (byte == 255) codes = 0;
        if (!pl[j].live) continue;
        reinterpret_cast<uint32_t *>(P.out)[first + j * 256 + threadIdx.x] = codes;
        // one lane of a block's four writes its scale byte; the row's last block fills its word up
        if ((pl[j].at & 3) == 0) {
            const uint32_t block = pl[j].at >> 2;
            uint8_t *words = P.scales + pl[j].row * P.words * 4;
            words[block] = (uint8_t)byte;
            if ((block + 1) * 4 == (uint32_t)P.unitsPerRow)
                for (uint32_t k = block + 1; k < (uint32_t)P.words * 4; ++k) words[k] = 127;
        }
    }
}

template <bool FP32>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(MxParams P) {
    const int64_t first = (int64_t)blockIdx.x * (256 * kUnits);
    const int64_t blockRow = first / P.unitsPerRow;
    const uint32_t blockAt = (uint32_t)(first - blockRow * P.unitsPerRow);
    Place pl[kUnits];
    uint32_t codes[kUnits], byte[kUnits];
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
        const uint32_t step = j * 256 + threadIdx.x;
        pl[j] = place_of(P, blockRow, blockAt, first + step, step);
        codes[j] = byte[j] = 0;
        if (pl[j].live) {
            codes[j] = reinterpret_cast<const uint32_t *>(P.in)[first + step];
            byte[j] = P.scales[pl[j].row * P.words * 4 + (pl[j].at >> 2)];
        }
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
        if (!pl[j].live) continue;
        const float scale = __uint_as_float(byte[j] == 0 ? 0x00400000u : byte[j] << 23);
        const bool nan = byte[j] == 255;
        const int64_t unit = first + j * 256 + threadIdx.x;
        if (FP32) {
            const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[j], scale, 0);
            const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[j], scale, 1);
            const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[j], scale, 2);
            const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[j], scale, 3);
            u32x4 lo = {__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y)};
            u32x4 hi = {__float_as_uint(c.x), __float_as_uint(c.y), __float_as_uint(d.x), __float_as_uint(d.y)};
            if (nan) lo = hi = u32x4{0x7fc00000u, 0x7fc00000u, 0x7fc00000u, 0x7fc00000u};
            store16<true>(P.out + unit * 32, lo);
            store16<true>(P.out + unit * 32 + 16, hi);
        } else {
            u32x4 o;
            o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[j], scale, 0));
            o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[j], scale, 1));
            o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[j], scale, 2));
            o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[j], scale, 3));
            if (nan) o = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
            store16<true>(P.out + unit * 16, o);
        }
    }
}

int64_t mx_blocks(const MxParams &P) { return (P.units + 256 * kUnits - 1) / (256 * kUnits); }

}  // namespace

hipError_t launch_mx_quantize(const MxParams &P, bool fp32, hipStream_t stream) {
    if (P.units == 0) return hipSuccess;
    if (mx_blocks(P) > INT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)mx_blocks(P));
    if (fp32)
        hipLaunchKernelGGL((mx_quantize_kernel<true>), grid, dim3(256), 0, stream, P);
    else
        hipLaunchKernelGGL((mx_quantize_kernel<false>), grid, dim3(256), 0, stream, P);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxParams &P, bool fp32, hipStream_t stream) {
    if (P.units == 0) return hipSuccess;
    if (mx_blocks(P) > INT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)mx_blocks(P));
    if (fp32)
        hipLaunchKernelGGL((mx_dequantize_kernel<true>), grid, dim3(256), 0, stream, P);
    else
        hipLaunchKernelGGL((mx_dequantize_kernel<false>), grid, dim3(256), 0, stream, P);
    return hipGetLastError();
}

}  // namespace epdc
