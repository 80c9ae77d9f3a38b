// Rows as int8 codes with one scale, for gfx950: of given rows, and of the
// gated activation's.
//
// scale = m / 127 (m the row's largest magnitude), code = rint(x / scale), both
// quotients rounded to fp32; a row with a NaN or an infinity: scale NaN, codes 0.
//
// Bound by memory.  A wave (short rows) or a block takes a row; its first
// elements stay in registers between the maximum and the codes, what is beyond
// them is read again (out of the cache).  32768 x 7168 bf16: 139-143 us, 5 TB/s.
// The activation's 32768 x 2048 take 118 us (2.9 TB/s), its instructions: by the
// time about 70 an element, of the exponential, the value, and three passes over
// the values; 2047 x 2048 13 us.
//
// The activation's codes are those of its values in 64 bits.  A 32-bit value a
// of it is within 2^-20 |a|: where a / scale is that near the border between
// two codes, or a that near the row's maximum, the value is taken again in 64
// bits (one element in 1000, and about one a row).
#include "expert_elems.h"

namespace epdc {
namespace {

constexpr uint32_t kInf = 0x7f800000u;

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The code of x, exactly as the quotient in fp32 gives it.
__device__ __forceinline__ int32_t code_of(float x, float scale) {
    const float q = rintf(x / scale);
    return (int32_t)fminf(fmaxf(q, -127.0f), 127.0f);
}

__device__ __forceinline__ void store_codes(uint8_t *row, int32_t unit, const int32_t (&c)[8]) {
    u32x2 v;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        v[i] = (uint32_t)(c[4 * i] & 255) | (uint32_t)(c[4 * i + 1] & 255) << 8 | (uint32_t)(c[4 * i + 2] & 255) << 16 |
               (uint32_t)(c[4 * i + 3] & 255) << 24;
    store8<false>(row + (int64_t)unit * 8, v);
}

// A row's scale from its largest magnitude (as bits; NaNs are above infinity).
__device__ __forceinline__ float scale_of(uint32_t most) {
    return most >= kInf ? __uint_as_float(0x7fc00000u) : __uint_as_float(most) / 127.0f;
}

template <bool FP32, int TEAM, int KEEP>
__global__ __launch_bounds__(256) void int_quantize_kernel(Int8Params P, DivMagic winDiv) {
    __shared__ uint32_t part[4];
    const int32_t lane = threadIdx.x % TEAM, units = P.cols / 8;
    for (int64_t row = (int64_t)blockIdx.x * (256 / TEAM) + threadIdx.x / TEAM; row < P.rows;
         row += (int64_t)gridDim.x * (256 / TEAM)) {
        if (P.rowCount) {
            const uint32_t w = div_by((uint32_t)row, winDiv);
            if ((int32_t)((uint32_t)row - w * (uint32_t)P.M) >= P.rowCount[w]) continue;
        }
        const uint8_t *x = P.x + (int64_t)row * P.cols * (FP32 ? 4 : 2);
        uint8_t *q = P.q + (int64_t)row * P.cols;
        Raw8<FP32> kept[KEEP];
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            if (lane + i * TEAM < units)
                kept[i] = load_raw8<FP32>(x, lane + i * TEAM);
            else
                kept[i] = Raw8<FP32>{};
        }
        uint32_t most = 0;
        auto highest = [&](const Eight &e) {
#pragma unroll
            for (int j = 0; j < 8; ++j) most = max(most, magnitude(e.v[j]));
        };
#pragma unroll
        for (int i = 0; i < KEEP; ++i) highest(to_eight<FP32>(kept[i]));
        for (int32_t unit = lane + KEEP * TEAM; unit < units; unit += TEAM) highest(to_eight<FP32>(load_raw8<FP32>(x, unit)));
        most = team_max<TEAM>(most, part);
        const float scale = scale_of(most);
        if (lane == 0) P.scales[row] = scale;
        const bool none = !(scale > 0.0f);
        auto codes = [&](const Eight &e, int32_t unit) {
            int32_t c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = none ? 0 : code_of(e.v[j], scale);
            store_codes(q, unit, c);
        };
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if (lane + i * TEAM < units) codes(to_eight<FP32>(kept[i]), lane + i * TEAM);
        for (int32_t unit = lane + KEEP * TEAM; unit < units; unit += TEAM) codes(to_eight<FP32>(load_raw8<FP32>(x, unit)), unit);
    }
}

// The activation's value, in 64 bits, rounded to fp32.  Out of line: few lanes get here.
__device__ __noinline__ float gate_exactly(float g, float u, float w) {
    const double s = 1.0 / (1.0 + exp(-(double)g));
    return (float)((double)g * s * (double)u * (double)w);
}

// A value's error in 32 bits: an exponential, a quotient and four products,
// below 12 half steps, so 2^-20 of it with room -- unless a factor leaves fp32's
// normal range on the way.  With the bounds below what is lost there is under
// 88 * 2^-126 * 2^30 * 2^15, 2^-27 of a code of a row whose maximum is above 2^-40.
constexpr float kClose = 0x1p-20f;
__device__ __forceinline__ bool plain_factors(float u, float w) { return fabsf(u) < 0x1p30f && w < 0x1p15f && w > 0x1p-15f; }

// A lane's first eight values stay in registers (the others are computed again)
// between three passes: the maximum in 32 bits; the maximum in 64 bits, of the
// values close to it; the codes.
template <bool FP32, int TEAM>
__global__ __launch_bounds__(256) void gate_int_kernel(GateParams P) {
    __shared__ uint32_t part[4];
    const RowRange rows = rows_of_groups(P.offsets, P.E, P.maxEntries);
    const int32_t lane = threadIdx.x % TEAM, units = P.F / 8;
    for (int64_t row = (int64_t)blockIdx.x * (256 / TEAM) + threadIdx.x / TEAM; row < rows.last;
         row += (int64_t)gridDim.x * (256 / TEAM)) {
        if (row < rows.first) continue;
        const uint8_t *h = P.h + (int64_t)row * P.F * (FP32 ? 8 : 4);
        const float w = P.entryWeight ? P.entryWeight[row] : 1.0f;
        struct Unit {
            Raw8<FP32> g, u;
            Eight a;
        };
        auto load = [&](int32_t unit) {
            Unit x{load_raw8<FP32>(h, unit), load_raw8<FP32>(h, units + unit), {}};
            const Eight g = to_eight<FP32>(x.g), u = to_eight<FP32>(x.u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // 1 / (1 + t) to a step
                const float t = expf(-fabsf(g.v[j])), large = __builtin_amdgcn_rcpf(1.0f + t);
                x.a.v[j] = g.v[j] * (g.v[j] >= 0.0f ? large : t * large) * u.v[j] * w;
            }
            return x;
        };
        auto each_value = [&](const Unit &x, auto &&f) {  // f(place, value in 32 bits, g, u)
            const Eight g = to_eight<FP32>(x.g), u = to_eight<FP32>(x.u);
#pragma unroll
            for (int j = 0; j < 8; ++j) f(j, x.a.v[j], g.v[j], u.v[j]);
        };
        Unit kept{};
        if (lane < units) kept = load(lane);
        auto each_unit = [&](auto &&f) {
            if (lane < units) f(kept, lane);
            for (int32_t unit = lane + TEAM; unit < units; unit += TEAM) f(load(unit), unit);
        };
        uint32_t most = 0;
        bool odd = false;  // factors beyond the bounds
        each_unit([&](const Unit &x, int32_t) {
            each_value(x, [&](int, float a, float, float u) {
                most = max(most, magnitude(a));
                odd |= !plain_factors(u, P.entryWeight ? fabsf(w) : 1.0f);
            });
        });
        most = team_max<TEAM>(most, part);
        // A row of odd factors, or of values beyond the middle of fp32's range: every value in 64 bits.
        const bool all = team_max<TEAM>(odd, part) != 0 || !(__uint_as_float(most) > 0x1p-40f && __uint_as_float(most) < 0x1p100f);
        const float near = __uint_as_float(most) * (1.0f - 2 * kClose);
        most = 0;
        each_unit([&](const Unit &x, int32_t) {
            each_value(x, [&](int, float a, float g, float u) {
                if (all || fabsf(a) >= near) most = max(most, magnitude(gate_exactly(g, u, w)));
            });
        });
        most = team_max<TEAM>(most, part);
        const float scale = scale_of(most);
        if (lane == 0) P.perEntry[row] = scale;
        const bool none = !(scale > 0.0f);
        const float over = 1.0f / scale;
        each_unit([&](const Unit &x, int32_t unit) {
            int32_t c[8];
            each_value(x, [&](int j, float a, float g, float u) {
                // Far enough from the border between two codes the quotient's last bits do not count: at 127 a value's
                // error is 2^-13 of a code, this product's another 2^-16.
                const float q = a * over, r = rintf(q);
                c[j] = (int32_t)fminf(fmaxf(r, -127.0f), 127.0f);
                if (all || fabsf(fabsf(q - r) - 0.5f) < 0x1p-11f) c[j] = none ? 0 : code_of(gate_exactly(g, u, w), scale);
            });
            store_codes(P.out + (int64_t)row * P.F, unit, c);
        });
    }
}

}  // namespace

hipError_t launch_int_quantize(const Int8Params &P, bool fp32, hipStream_t stream) {
    const DivMagic div = div_magic((uint32_t)P.M);
    const bool wave = P.cols <= 1024;
    const dim3 grid((uint32_t)min(wave ? (P.rows + 3) / 4 : P.rows, kMostBlocks));
    if (wave && fp32)
        hipLaunchKernelGGL((int_quantize_kernel<true, 64, 2>), grid, dim3(256), 0, stream, P, div);
    else if (wave)
        hipLaunchKernelGGL((int_quantize_kernel<false, 64, 2>), grid, dim3(256), 0, stream, P, div);
    else if (fp32)
        hipLaunchKernelGGL((int_quantize_kernel<true, 256, 4>), grid, dim3(256), 0, stream, P, div);
    else
        hipLaunchKernelGGL((int_quantize_kernel<false, 256, 4>), grid, dim3(256), 0, stream, P, div);
    return hipGetLastError();
}

hipError_t launch_gate_int(const GateParams &P, bool fp32, hipStream_t stream) {
    const bool wave = P.F <= 512;
    const dim3 grid((uint32_t)min((int64_t)(wave ? ceil_div(P.maxEntries, 4) : P.maxEntries), kMostBlocks));
    if (wave && fp32)
        hipLaunchKernelGGL((gate_int_kernel<true, 64>), grid, dim3(256), 0, stream, P);
    else if (wave)
        hipLaunchKernelGGL((gate_int_kernel<false, 64>), grid, dim3(256), 0, stream, P);
    else if (fp32)
        hipLaunchKernelGGL((gate_int_kernel<true, 256>), grid, dim3(256), 0, stream, P);
    else
        hipLaunchKernelGGL((gate_int_kernel<false, 256>), grid, dim3(256), 0, stream, P);
    return hipGetLastError();
}

}  // namespace epdc
