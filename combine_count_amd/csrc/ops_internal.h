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

// The routing's kernel for a shape.
struct RoutePlan {
    int32_t lanes;    // of a token: 16 or 64 (the fast form; the gradient's form of four tokens a wave), 0: the general form
    int32_t perLane;  // experts of a lane
    bool inRow;       // a lane's experts lie in a row, one load; else lane, lane + lanes, ...
};

// Up to this many tokens a whole wave takes a token of 256 experts: fewer
// instructions one behind the other, where there are waves for it (8 groups,
// biased, bf16; 8 / 1024 / 2048 / 4096 tokens: 5.5 / 6.4 / 6.8 / 8.1 us against
// 5.8 / 7.1 / 7.2 / 7.3 with four tokens a wave).
constexpr int32_t kWaveTokens = 2048;

inline RoutePlan plan_route(int32_t E, int32_t K, int32_t G, int32_t keep, int32_t T, bool softmax, bool biased, bool aligned) {
    const bool limited = keep < G, inRow = (E == 64 || E == 128 || E == 256) && aligned;
    // The fast form needs a choice value that 32 bits give nearly (a biased
    // softmax's hangs on a sum over all experts), a lane for one more than K, and
    // groups that are whole lanes.
    const bool fast = !(softmax && biased) && (!limited || (inRow && 16 % G == 0));
    if (fast && inRow && E == 256 && K < 64 && T <= kWaveTokens) return RoutePlan{64, 4, true};
    if (fast && E <= 256 && K < 16) return RoutePlan{16, E <= 64 ? 4 : E <= 128 ? 8 : 16, inRow};
    if (fast && !limited && K < 64) return RoutePlan{64, E <= 256 ? 4 : E <= 512 ? 8 : 16, false};
    return RoutePlan{0, E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 4 : E <= 512 ? 8 : 16, false};
}

// aligned: logits and dLogits at 16-byte borders.
inline RoutePlan plan_route_grad(int32_t E, int32_t K, bool aligned) {
    if ((E == 64 || E == 128 || E == 256) && K <= 16 && aligned) return RoutePlan{16, E / 16, true};
    return RoutePlan{0, E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 4 : E <= 512 ? 8 : 16, false};
}

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

// The product's kernels: weights streamed into registers in tiles of 16 or 64
// entries, tiles of 128 x 128 (with 64-bit offsets of the rows: wide) or
// 256 x 256 through LDS.
enum ProductForm { kProductStream16, kProductStream64, kProductTiles128, kProductTiles128Wide, kProductTiles256 };

// Which kernel, from the entries that can occur (the groups' sizes are known
// on the device only).  Times in us, 4096 columns unless stated:
//   * 256x256 tiles move the fewest operand bytes per product, and take over
//     where the mean group fills a good part of one and there are tiles for
//     two rounds of all CUs: h7168, 32 experts, 3000 / 4096 / 6144 / 32768
//     entries 148 / 151 / 158 / 542 against 126 / 165 / 194 / 693 with
//     128x128; 8 experts, 4096 entries (320 tiles) 100 against 94;
//   * streamed weights where experts have a few entries and rows are long:
//     h7168, 32 experts, 64 / 32 / 16 entries 79 / 54 / 27 against 91 / 71 / 33
//     with 128x128 tiles (at h4096 48 against 43, h2048 37 against 27: the
//     block's fixed cost);
//   * and where 128x128 tiles would leave most CUs idle: h7168, one expert, 8 /
//     32 / 64 entries 9 / 10 / 16 against 19; 8 experts, 8 entries 13 against 25;
//     2 experts, 64 entries 14 (64-entry tiles; 20 with 16-entry ones) against 24;
//     but 8 experts, 128 entries 32 against 28.
inline ProductForm plan_product(int32_t E, int32_t N, int32_t H, int32_t maxEntries, int32_t numRows) {
    const int32_t mean = ceil_div(maxEntries, E);
    const int64_t groups = E < maxEntries ? E : maxEntries;
    const int64_t tiles128 = (maxEntries / 128 + groups) * ceil_div(N, 128);
    const int64_t tiles256 = (maxEntries / 256 + groups / 2) * ceil_div(N, 256);
    if ((mean <= 4 && H >= 6144) || (mean <= 8 && tiles128 <= 288) || (mean <= 24 && tiles128 <= 160)) return kProductStream16;
    if (tiles128 <= 160) return kProductStream64;
    if ((int64_t)numRows * (H / 2) > 0xf0000000ll) return kProductTiles128Wide;
    return mean >= 96 && tiles256 >= 512 ? kProductTiles256 : kProductTiles128;
}

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
