// Kernel parameters and launchers of the operators next to dispatch and
// combine: routing (route.hip), fp4x2 quantisation (mx.hip), grouping by
// expert (group.hip) and the experts' product (product.hip).  Not part of
// the C ABI.
#pragma once

#include "epdc_internal.h"

namespace epdc {

struct RouteParams {
    int32_t E, K, T;
    int32_t G, keep, groupTop;  // groups, groups kept per token, best values summed per group
    int32_t perGroup;           // E / G
    int32_t softmax, renorm;    // else sigmoid
    float scale;
    const void *logits;      // [T][E] bf16 or fp32
    const float *bias;       // [E] or NULL
    int32_t *expertIds;      // [T][K]
    float *weights;          // [T][K]
};

struct RouteGradParams {
    int32_t E, K, T;
    int32_t softmax, renorm;
    float scale;
    const void *logits;
    const int32_t *expertIds;
    const float *dWeights;
    void *dLogits;
};

// Rows of W windows of M rows; with rowCount only rows r < rowCount[w].
struct MxParams {
    int64_t units;        // rows * cols / 8: 8 elements are one thread's share
    int32_t unitsPerRow;  // cols / 8
    int32_t M;
    int32_t words;        // scale words per row
    DivMagic rowDiv;      // by unitsPerRow
    DivMagic winDiv;      // by M
    const int32_t *rowCount;
    const uint8_t *in;    // x, or q
    uint8_t *out;         // q, or the values
    uint8_t *scales;
};

struct GroupParams {
    int32_t W, M, K, Epr;
    int32_t rank;            // -1: window w is grouped over its own PE's experts
    int32_t tileRows;        // rows of a tile; a tile lies in one window
    int32_t tilesPerWindow;
    DivMagic windowDiv;      // by M * K
    const int32_t *expertIds;
    const float *weights;
    const int32_t *recvCount;
    int32_t *offsets;
    int32_t *entryRow;
    float *entryWeight;
    int32_t *entryOf;
    int32_t *hist;           // scratch: [W * tilesPerWindow][Epr], then the totals of the large form
};

// About 2048 slots a tile: enough rows per block to fill its waves, few
// enough tiles that a block can sum their counts itself.
constexpr int kGroupTileSlots = 2048;
// Launches of up to this many slots count all of them in every block (one
// launch; 8 windows of 64 rows x 8: 8.5 us against 9.9, of 128: 11.7 against 10.7).
constexpr int64_t kGroupLocalSlots = 4096;
// Launches of up to this many published words sum them in every block; more
// go through scan launches.
constexpr int64_t kGroupSelfWords = 32768;
inline int32_t group_tile_rows(int32_t K) { return K >= kGroupTileSlots ? 1 : kGroupTileSlots / K; }
inline int32_t group_tiles_per_window(int32_t M, int32_t K) { return ceil_div(M, group_tile_rows(K)); }

struct ProductParams {
    int32_t E, N, H;          // experts, output columns, elements per row
    int32_t maxEntries, numRows;
    int32_t rowBytes;         // H / 2
    int32_t words;            // scale words per row
    const uint8_t *rows;
    const uint8_t *rowScales;
    const int32_t *offsets;
    const int32_t *entryRow;
    const float *entryWeight;
    const uint8_t *weights;
    const uint8_t *weightScales;
    void *out;
};

template <int I>
struct Const {
    static constexpr int value = I;
};
// f(Const<0>), ..., f(Const<N-1>): indices that are constants in f.
template <int N, int I = 0, class F>
__device__ __forceinline__ void each(F &&f) {
    if constexpr (I < N) {
        f(Const<I>{});
        each<N, I + 1>(f);
    }
}

inline __device__ uint32_t div_by(uint32_t n, DivMagic d) {
    const uint32_t t = __umulhi(n, d.magic);
    return (t + ((n - t) >> d.sh1)) >> d.sh2;
}

// fp32 -> bf16 bits, round to nearest, ties to even; NaN stays a quiet NaN.
__device__ __forceinline__ uint32_t bf16_rne(float f) {
    uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return (u >> 16) | 0x40u;
    u += 0x7fffu + ((u >> 16) & 1u);
    return u >> 16;
}

// Orders this wave's LDS accesses: the hardware keeps a wave's LDS
// operations in order, so only the compiler has to be told.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

hipError_t launch_route(const RouteParams &p, bool fp32, hipStream_t stream);
hipError_t launch_route_grad(const RouteGradParams &p, bool fp32, hipStream_t stream);
hipError_t launch_mx_quantize(const MxParams &p, bool fp32, hipStream_t stream);
hipError_t launch_mx_dequantize(const MxParams &p, bool fp32, hipStream_t stream);
int64_t group_scratch_words(int32_t W, int32_t M, int32_t K, int32_t Epr);
hipError_t launch_group(const GroupParams &p, hipStream_t stream);
hipError_t launch_product(const ProductParams &p, bool out32, hipStream_t stream);

}  // namespace epdc
