// Kernel parameters and launchers of the operators next to dispatch and
// combine: routing (route.hip), fp4x2 quantisation (mx.hip), grouping by
// expert (group.hip), the experts' product (product.hip), and the experts in
// bf16 and int8 (product_dense.h, gate.hip, int8.hip).  Not part of the C ABI.
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

// A product of bf16 or int8 rows and its gradients.
struct DenseParams {
    int32_t E, N, H;          // experts, output columns, elements per row
    int32_t maxEntries;
    int32_t numRows;          // of rows (the rows' gradient: of dOut)
    int32_t numOutRows;       // of dOut (the weights' gradient)
    const uint8_t *rows;      // [numRows][H] (the rows' gradient: dOut [numRows][N])
    const float *rowScales;   // [numRows], int8
    const int32_t *offsets;
    const int32_t *entryRow;
    const float *entryWeight;
    const uint8_t *weights;   // [E][N][H]
    const float *weightScales;  // [E][N], int8
    const uint8_t *dOut;      // [numOutRows][N], the weights' gradient
    const int32_t *outRow;
    const uint8_t *base;      // [E][N][H] of the output's type, or NULL
    uint8_t *out;
};
// out = rows . weights^T; dRows = dOut . weights; dWeights = dOut^T . rows
enum DenseKind { kDenseProduct, kDenseRowsGrad, kDenseWeightsGrad };

// Their kernels: weights streamed into registers for tiles of 16 or 64 entries
// (the product), tiles of 128 x 128 or 256 x 256 of the output through LDS.
enum DenseForm { kDenseStream16, kDenseStream64, kDenseTiles128, kDenseTiles256 };

// Which kernel, from the entries that can occur (the groups' sizes are known on
// the device only).  Times in us, bf16 / int8, groups of equal size, weights from
// memory (one to four experts' stay in the cache from call to call where nothing
// else runs: tiles then take 76 / 42 for one expert, the streaming forms as here),
// 7168 -> 4096 unless stated:
//   * weights streamed where 128x128 tiles would leave CUs idle and experts have
//     few entries: one expert, 16 entries 28 / 16, 64 entries 49 / 27 against 106 /
//     57 with tiles; 8 experts, 64 entries 98 / 51 against 120 / 64; 9 experts, 72
//     entries 122 / 64 against 125 / 68 (10 experts, 80 entries, beyond the border:
//     125 / 65 against 129 / 69); 16 experts, 128 entries 200 / 102 against 159 / 86;
//     32 experts, 64 entries 352 / 179 against 308 / 162.  Tiles of 64 entries beyond
//     16 an expert: 2 experts, 64 entries 39 / 22 against 51 / 28 with 16; 4 experts,
//     128 entries 74 / 39 against 97 / 51 (128x128: 111 / 59); but 8 experts, 256
//     entries 143 / 73 against 121 / 65 with 128x128; one expert, 256 entries 87 / 46
//     against 108 / 58, 512 entries 173 / 89 against 107 / 57;
//   * 256x256 tiles where the mean group fills a good part of one and there is
//     one for every CU: 8 experts, 4096 entries 220 / 122 against 284 / 152, 2048
//     entries 204 / 109 against 162 / 88; 32 experts, 4096 entries 414 / 225 against
//     384 / 211; 32 experts, 2048 -> 7168, 8192 entries 290 / 157 against 321 / 186;
//     one expert, 8192 entries 387 / 205 against 485 / 267, 2048 entries 173 / 94
//     against 130 / 72.  Groups whose sizes differ (entries dealt out at random) need
//     more tiles of 128 rows, and the border lies lower: 8 experts, 2048 entries 203 /
//     110 with 256x256 against 250 / 130, 32 experts, 4096 entries 421 / 229 against
//     512 / 266, both beyond what the rule takes; 8 experts, 4096 entries 376 / 193
//     against 368 / 192;
//   * the weights' gradient likewise (its tiles are all there, whatever the
//     groups), bf16 rows: 16 experts, 1024 x 1024, 256 tiles: 16384 / 333 entries 41 /
//     16.6 against 49 / 17.4; 32 experts, 7168 -> 4096, 4096 entries, fp32 764 against
//     1071.
inline DenseForm plan_dense(DenseKind kind, int32_t E, int32_t N, int32_t H, int32_t maxEntries) {
    const int32_t columns = kind == kDenseProduct ? N : H;
    if (kind == kDenseWeightsGrad)
        return (int64_t)E * ceil_div(N, 256) * ceil_div(H, 256) >= 256 ? kDenseTiles256 : kDenseTiles128;
    const int32_t mean = ceil_div(maxEntries, E);
    const int64_t groups = E < maxEntries ? E : maxEntries;
    const int64_t tiles128 = (maxEntries / 128 + groups) * ceil_div(columns, 128);
    const int64_t tiles256 = (maxEntries / 256 + groups / 2) * ceil_div(columns, 256);
    if (kind == kDenseProduct && mean <= 16 && tiles128 <= 288) return kDenseStream16;
    if (kind == kDenseProduct && ((mean <= 128 && tiles128 <= 192) || (mean <= 256 && tiles128 <= 96))) return kDenseStream64;
    return mean >= 192 && tiles256 >= 256 ? kDenseTiles256 : kDenseTiles128;
}

struct GateParams {
    int32_t E, F, maxEntries;
    const uint8_t *h;         // [maxEntries][2 F]
    const int32_t *offsets;   // or NULL
    const float *entryWeight;
    const uint8_t *dOut;      // [maxEntries][F]
    uint8_t *out;             // [maxEntries][F]; the gradient: dH [maxEntries][2 F]; int8 codes
    float *perEntry;          // the gradient: dEntryWeight or NULL; int8: scales
};

struct Int8Params {
    int32_t M, cols;          // rows per window
    int64_t rows;
    const int32_t *rowCount;
    const uint8_t *x;
    uint8_t *q;
    float *scales;
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
hipError_t launch_dense_linear(const DenseParams &p, DenseForm form, bool out32, hipStream_t stream);
hipError_t launch_dense_linear_int(const DenseParams &p, DenseForm form, bool out32, hipStream_t stream);
hipError_t launch_dense_rows_grad(const DenseParams &p, DenseForm form, bool out32, hipStream_t stream);
hipError_t launch_dense_weights_grad(const DenseParams &p, DenseForm form, bool out32, hipStream_t stream);
hipError_t launch_gate(const GateParams &p, bool fp32, bool out32, hipStream_t stream);
hipError_t launch_gate_grad(const GateParams &p, bool fp32, bool out32, hipStream_t stream);
hipError_t launch_gate_int(const GateParams &p, bool fp32, hipStream_t stream);
hipError_t launch_int_quantize(const Int8Params &p, bool fp32, hipStream_t stream);

}  // namespace epdc
