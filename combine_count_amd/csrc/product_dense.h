// The products of bf16 and int8 rows with the experts' weights, and the bf16
// product's two gradients, for gfx950: over a group's entries i
//   product           out[i][n]   = sum_h rows[r_i][h] W[n][h]
//   rows' gradient    dRows[i][h] = sum_n dOut[r_i][n] W[n][h]
//   weights' gradient dW[n][h]    = sum_i dOut[o_i][n] rows[r_i][h]
//
// Tiles of 256 x 256 or 128 x 128 of the output, through LDS, with
// v_mfma_f32_32x32x16_bf16 (v_mfma_i32_32x32x32_i8: the same bytes a lane);
// plan_dense chooses.  The kernel's time, median (least) of 40 passes under load:
// 32768 entries of 32 experts, 7168 -> 4096, groups of different sizes: bf16 1.76
// (1.73) ms, 1.09 PFLOP/s, int8 0.87 (0.85) ms, 2.2 POP/s (a loop of the
// instruction alone 1.78 and 3.5), the matrix cores busy 71% of the time at a
// clock of 1.65 GHz; one dense product of 8192^3 1.36 PFLOP/s.  Rows' gradient,
// 16384 entries, 7168 -> 2048: 0.56 (0.53) ms.  Weights' gradient, 16384 entries,
// 4096 x 7168: 1.20 (1.18) ms, bound by the results' stores between tiles of eight
// steps (0.95 without them).  64 entries of 32 experts, bound by the weights: 283
// (272) us, 5.8 TB/s.  (Of 20 passes that begin on an idle card, whose clocks are
// still rising, the same kernels take up to a seventh longer.)
#pragma once

#include "tiles.h"

namespace epdc {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_dword __attribute__((ext_vector_type(4), aligned(4)));  // 16 bytes at 4-byte alignment

// The sums of 32 x 32 products stay in accumulation registers of their own,
// named here (fragment f: a16f .. a16f + 15): the compiler's own allocation of
// 256 of them moved them about or spilled where the kernel has several bodies.
// It sees them as overwritten in every half of a step (hold_sums), so that it
// keeps nothing there; that it does not use them in between either is checked on
// the built code.  It does not see the matrix instruction: its operands must not
// come from a vector instruction just before it, and its sums are read behind
// mfma_done().
#define EPDC_A10(n) "a" #n "0", "a" #n "1", "a" #n "2", "a" #n "3", "a" #n "4", "a" #n "5", "a" #n "6", "a" #n "7", "a" #n "8", "a" #n "9"
#define EPDC_SUMS64 \
    "a0", "a1", "a2", "a3", "a4", "a5", "a6", "a7", "a8", "a9", EPDC_A10(1), EPDC_A10(2), EPDC_A10(3), EPDC_A10(4), EPDC_A10(5), "a60", "a61", "a62", "a63"
#define EPDC_SUMS256 \
    EPDC_SUMS64, "a64", "a65", "a66", "a67", "a68", "a69", EPDC_A10(7), EPDC_A10(8), EPDC_A10(9), EPDC_A10(10), EPDC_A10(11), EPDC_A10(12), EPDC_A10(13), \
        EPDC_A10(14), EPDC_A10(15), EPDC_A10(16), EPDC_A10(17), EPDC_A10(18), EPDC_A10(19), EPDC_A10(20), EPDC_A10(21), EPDC_A10(22), EPDC_A10(23), EPDC_A10(24), \
        "a250", "a251", "a252", "a253", "a254", "a255"
template <int ALL>
__device__ __forceinline__ void hold_sums() {
    if constexpr (ALL == 16)
        asm volatile("" : : : EPDC_SUMS256);
    else
        asm volatile("" : : : EPDC_SUMS64);
}
// Fragment F: += a . b, or with FIRST = a . b.
template <int F, bool FIRST, bool INT8>
__device__ __forceinline__ void mfma_sums(u32x4 a, u32x4 b) {
    if constexpr (INT8 && FIRST)
        asm volatile("v_mfma_i32_32x32x32_i8 a[%2:%3], %0, %1, 0" : : "v"(a), "v"(b), "n"(F * 16), "n"(F * 16 + 15));
    else if constexpr (INT8)
        asm volatile("v_mfma_i32_32x32x32_i8 a[%2:%3], %0, %1, a[%2:%3]" : : "v"(a), "v"(b), "n"(F * 16), "n"(F * 16 + 15));
    else if constexpr (FIRST)
        asm volatile("v_mfma_f32_32x32x16_bf16 a[%2:%3], %0, %1, 0" : : "v"(a), "v"(b), "n"(F * 16), "n"(F * 16 + 15));
    else
        asm volatile("v_mfma_f32_32x32x16_bf16 a[%2:%3], %0, %1, a[%2:%3]" : : "v"(a), "v"(b), "n"(F * 16), "n"(F * 16 + 15));
}
// Sum V of fragment F, as it lies in the register.
template <int F, int V>
__device__ __forceinline__ uint32_t read_sum() {
    uint32_t x;
    asm volatile("v_accvgpr_read_b32 %0, a[%1]" : "=v"(x) : "n"(F * 16 + V));
    return x;
}

// Four bf16 of a column of a 4 x 16 block in LDS (rows of the block 8 bytes at
// a lane's address, four lanes a row): lane l of 16 gets column l.
__device__ __forceinline__ u32x2 read_turned(const uint8_t *p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p));
}

// 16 bytes per lane (or 4) from memory into LDS at the address lds, the same in
// all lanes, + lane * 16 (4).  In assembly, so that the compiler does not see a
// write to LDS under way: it would hold back reads of other parts of it until
// every load has arrived.  Only the waits written out here (meet) order them.
// They set m0, which nothing else in these kernels uses.
__device__ __forceinline__ uint32_t lds_address(const void *lds) {
    return uniform((int32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t *)lds);
}
__device__ __forceinline__ const uint8_t *uniform_pointer(const uint8_t *p) {
    return reinterpret_cast<const uint8_t *>(uniform64(reinterpret_cast<uint64_t>(p)));
}
template <int AT>
__device__ __forceinline__ void load_lds16_unseen(const uint8_t *src, uint32_t lds) {  // to lds + AT
    asm volatile("s_add_u32 m0, %0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(lds), "v"(src), "n"(AT) : "scc");
}
template <int AT>
__device__ __forceinline__ void load_lds16_unseen(const uint8_t *base, uint32_t off, uint32_t lds) {  // base the same in all lanes
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base), "n"(AT)
                 : "scc");
}
__device__ __forceinline__ void load_lds4_unseen(const int32_t *src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" : : "s"(lds), "v"(src));
}

__device__ u32x4 zero_piece;  // what is loaded in place of pieces that do not exist; never written

// Exchanges b's even rows of 16 lanes with a's odd ones, and b's lower 32 lanes with a's upper ones.
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// For the compiler: code of a tile's ends lies outside the loop over its steps.
__device__ __forceinline__ bool rarely(bool b) { return __builtin_expect(b, 0); }

// Where a tile of the output lies: expert, entries [lo, hi) of its group (of
// the tile, but for the weights' gradient), rows from r0, columns from c0.
struct DenseTile {
    int32_t e, lo, hi, r0, c0;
};

// A BM x BN tile of the output by four waves, half its columns and every other
// 32 of its rows each, in 32 x 32 fragments; the output's columns are the
// instruction's rows and its rows the instruction's columns, so a lane ends with
// runs of 8 consecutive columns of one row.  A tile of fewer rows takes the
// fragments that hold them only, and a group's rows are dealt out evenly over
// its tiles, 64 by 64 (1024 entries of an expert on average: an eighth of the
// products of whole tiles would be of rows that do not exist).
//
// The summed index goes in steps of 128 bytes of it (64 bf16, 128 int8) through
// two pairs of places in LDS, loaded by the memory pipeline itself.  A step is
// two halves; the operands of a half are read into registers during the half
// before:
//     products of half 0 | read half 1 of step k
//     wait: step k+1 has arrived (requested one whole step ago); barrier
//     products of half 1 | request step k+2 into step k's places,
//                        | read half 0 of step k+1
// (Into the registers of products just issued instead, every read waits for
// them: a fifth slower.  A fifth place, for the rows of step k+3: no gain.)
// The steps of a block's tiles follow one another without a gap: behind a
// tile's last step come the next tile's first (a stride of the grid further),
// requested while the last ones are computed; a tile's results are stored with
// them under way.  A tile has two steps at least (of zeros, if need be).  What a
// tile's begin and end need lies outside the loop over its steps: with it in
// between, the loop's instructions come late (a quarter slower).
//
// An operand whose summed index runs along its rows in memory lies in LDS in
// rows of 128 bytes, their 16-byte pieces at piece ^ row / 2 % 8, so that the 16
// lanes that read one piece of 16 rows spread over the 256 bytes of the banks.  The others (turned: the rows' gradient's weights, both of the
// weights' gradient) lie as they do in memory, a row of BX elements per value
// of the summed index, 64 of them a step, and are turned over as they are
// read, four at a time; their 64-byte chunks lie at chunk ^ s, s of the row's
// index, so that the eight rows of a read spread over the banks.
template <DenseKind KIND, bool INT8, int BM, int BN, bool OUT32>
__global__ __launch_bounds__(256, BM *BN > 128 * 128 ? 1 : 2) void dense_tile_kernel(DenseParams P) {
    constexpr bool kTurnedC = KIND != kDenseProduct, kTurnedR = KIND == kDenseWeightsGrad;
    constexpr int ES = INT8 ? 1 : 2;            // bytes of an element
    constexpr int FR = BM / 64, FC = BN / 64;   // fragments of a wave
    constexpr int LR = BM / 32, LC = BN / 32;   // LDS loads of a wave per step (1 KB each)
    static_assert(BM == BN, "the places in LDS hold either operand");
    constexpr int kPlace = BM * 128;
    __shared__ __attribute__((aligned(16))) uint8_t ring[4 * kPlace];  // rows and columns of a step, those of the next
    // The weights' gradient: rows of a step's entries (of dOut, of rows), of four steps that follow one another.
    __shared__ int32_t list[4][2][64];
    // The others: of the rows of this tile and the next, the entry's weight, its scale, and whether it has a row.
    struct RowInfo {
        float factor, scale;
        int32_t there;
    };
    __shared__ RowInfo rowInfo[KIND == kDenseWeightsGrad ? 1 : 2][KIND == kDenseWeightsGrad ? 1 : BM];
    const int32_t C = KIND == kDenseProduct ? P.N : P.H;  // the output's columns
    const int32_t RT = ceil_div(P.N, BM), CT = ceil_div(C, BN);
    const int32_t rowOut = C * (OUT32 ? 4 : 2);
    const int32_t kBytes = KIND == kDenseProduct ? P.H * ES : P.N * ES;  // of a row of the summed index (not the weights' gradient)
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wr = (wave & 1) * 32, wc = (wave >> 1) * (BN / 2);  // its fragments' rows from wr, 64 apart
    // The lane again, opaque: what is computed from it is computed there, not kept in registers from tile to tile.
    auto fresh = [&] {
        int l = lane;
        asm volatile("" : "+v"(l));
        return l;
    };
    const uint8_t *const zero = reinterpret_cast<const uint8_t *>(&zero_piece);

    // ---- tiles
    Groups groups;
    if constexpr (KIND == kDenseWeightsGrad) {
        int32_t least = P.maxEntries;
        load_groups<BM>(P, 0, least, groups);  // all there are, where they are 64 at most
    } else {
        groups = count_tiles<BM>(P, CT);
    }
    auto find = [&](int32_t b) {
        DenseTile t{-1, 0, 0, 0, 0};
        if constexpr (KIND == kDenseWeightsGrad) {
            // An XCD (block b % 8) takes 32 tiles in a row of every 256: those that run on it together share operands
            // in its L2, and every XCD has its part of every expert, whose groups differ in length.
            const int32_t i = b >> 3, tiles = RT * CT;
            const int64_t total = (int64_t)P.E * tiles;
            const int32_t run = (int32_t)min((total + 7) / 8, (int64_t)32);
            const int64_t at = ((int64_t)(i / run) * 8 + (b & 7)) * run + i % run;
            if (at >= total) return t;
            const int32_t e = (int32_t)(at / tiles), rest = (int32_t)(at - (int64_t)e * tiles);
            if (P.E > 64) {
                int32_t least = P.maxEntries;
                for (int32_t e0 = (P.E - 1) & ~63; e0 >= (e & ~63); e0 -= 64) load_groups<BM>(P, e0, least, groups);
            }
            const int32_t size = ceil_div(RT, max(RT >> 2, 1));  // row tiles of a band
            const int32_t band = rest / (size * CT), rows = min(size, RT - band * size), r = rest - band * size * CT;
            const int32_t c = r / rows;
            t = DenseTile{uniform(e), __builtin_amdgcn_readlane(groups.lo, e & 63), __builtin_amdgcn_readlane(groups.hi, e & 63),
                          uniform((band * size + r - c * rows) * BM), uniform(c * BN)};
        } else {
            const PlaceOf a = find_place<BM, BN>(P, groups, CT, b);
            if (a.e < 0) return t;
            const int64_t pairs = ceil_div((int64_t)a.hi - a.lo, 64);  // of fragments of the group, dealt out over its tiles
            const int32_t first = (int32_t)(pairs * a.m / a.tiles), end = (int32_t)(pairs * (a.m + 1) / a.tiles);
            t = DenseTile{a.e, a.lo + first * 64, (int32_t)min((int64_t)a.hi, a.lo + (int64_t)end * 64), 0, a.n0};
        }
        return DenseTile{uniform(t.e), uniform(t.lo), uniform(t.hi), uniform(t.r0), uniform(t.c0)};
    };
    auto steps_of = [&](const DenseTile &t) {
        if constexpr (KIND == kDenseWeightsGrad)
            return max((t.hi - t.lo + 63) / 64, 2);
        else
            return max((kBytes + 127) / 128, 2);
    };

    // ---- requests: tile Q, its step kq next; behind it tile next
    int32_t b = blockIdx.x;
    DenseTile next = find(b), Q{-1, 0, 0, 0, 0};
    if (next.e < 0) return;
    int32_t kq = 0, stepsQ = 0;
    // Rows along the summed index: this lane's rows, its columns' offsets from the tile's first, and the place in a row
    // (of even and odd loads) that it requests.
    uint32_t rowi[kTurnedR ? 1 : LR];
    uint32_t colo[kTurnedC ? 1 : LC];
    const int piece = ((lane & 7) ^ (lane >> 4)) * 16;  // of a step, in even loads (in odd ones ^ 64)
    const uint8_t *placeR[2] = {nullptr, nullptr};
    uint32_t placeC[2] = {0, 0};
    const uint8_t *stepBase = nullptr;  // columns that are not gathered: from where this step's are requested
    // Of entry wave * (BM/4) + lane: row and weight in the next tile, on their way, and what is known of it in tile Q.
    int32_t entryRow = -1;
    float entryWeight = 1.0f;
    RowInfo infoQ{};
    // Turned rows: lanes of a row of BX elements, rows of a load, and the 16-byte piece that this lane requests.
    constexpr int kLanesR = BM / 8, kPerR = 64 / kLanesR, kLanesC = BN / 8, kPerC = 64 / kLanesC;
    constexpr int kSwR = BM == 256 ? 4 : 1, kSwC = BN == 256 ? 4 : 1;  // swizzles of a wave's loads
    uint32_t turnedC[kTurnedC ? kSwC : 1];
    const uint8_t *fromR[kTurnedR ? kSwR : 1], *fromC[kTurnedR ? kSwC : 1];  // gathered: of row 0
    const uint8_t *src[kTurnedR ? LR + LC : 1];                             // and of the step's rows
    // offset of the piece in the tile's part of a row, by the load's swizzle; behind the row's end the last piece
    auto turned_piece = [&](auto bx, int s, int32_t left) {
        constexpr int BX = decltype(bx)::value;
        const int ln = fresh(), p = ln & (BX / 8 - 1);
        const int sw = BX == 256 ? ((s & 1) * 2 + (ln >> 5)) | (s >> 1) << 2 : ln >> 4;
        return (uint32_t)min((p ^ (sw << 2)) * 16, left * 2 - 16);
    };
    int32_t listR = 0, listC = 0;  // the weights' gradient: rows of entry `lane` of the next step, as listed
    int32_t idxR = 0, idxC = 0;    // and of the step that is requested
    uint64_t dead = 0;             // its entries that are none
    uint32_t slot = 0;             // its place among all steps, % 4 its lists' place
    const uint8_t *colBase = nullptr;
    auto fetch_entry = [&](const DenseTile &t) {  // product, rows' gradient
        const int32_t ent = t.lo + wave * (BM / 4) + (fresh() & (BM / 4 - 1));
        entryRow = -1;
        if (t.e >= 0 && ent < t.hi) {
            entryRow = P.entryRow ? P.entryRow[ent] : ent;
            if (P.entryWeight) entryWeight = P.entryWeight[ent];
        }
    };
    // Weights' gradient: the lists of step k of a tile, on their way into a place; wave 0 asks for dOut's, wave 1 for rows'.
    auto request_lists = [&](const DenseTile &t, int32_t k, uint32_t place) {
        const int32_t *from = wave == 0 ? P.outRow : P.entryRow;
        if (wave >= 2 || !from || t.e < 0) return;
        const int32_t at = k * 64 + lane;
        if (at < t.hi - t.lo) load_lds4_unseen(from + t.lo + at, lds_address(list[place & 3][wave]));
    };
    auto read_lists = [&](uint32_t place) {
        if (P.outRow) listR = list[place & 3][0][lane];
        if (P.entryRow) listC = list[place & 3][1][lane];
    };
    // Tile Q becomes `next`, or stays where there is none: what is requested then is not used.  What is known of Q's
    // rows, now the tile that is computed, goes to LDS.
    int turns = 0;
    auto turn_to_next = [&] {
        kq = 0;
        if constexpr (KIND != kDenseWeightsGrad) {
            const int row = wave * (BM / 4) + fresh();
            if (row < (wave + 1) * (BM / 4)) rowInfo[turns & 1][row] = infoQ;
        }
        ++turns;
        if (next.e < 0) {
            Q.e = -1;
            stepsQ = INT32_MAX;
            return;
        }
        Q = next;
        stepsQ = steps_of(Q);
        if constexpr (KIND != kDenseWeightsGrad) {
            const int ln = fresh();
            const bool there = (uint32_t)entryRow < (uint32_t)P.numRows;
            const int32_t row = there ? entryRow : 0;  // an entry without a row: any row, and zeros stored
#pragma unroll
            for (int i = 0; i < LR; ++i) rowi[i] = (uint32_t)__shfl(row, i * 8 + (ln >> 3));
            infoQ = RowInfo{entryWeight, 0.0f, there};
            if constexpr (INT8) {
                if (there) infoQ.scale = P.rowScales[row];
            }
        }
        if constexpr (KIND == kDenseProduct) {
            const int ln = fresh();
            colBase = P.weights + ((int64_t)Q.e * P.N + Q.c0) * kBytes;
#pragma unroll
            for (int i = 0; i < LC; ++i) colo[i] = (uint32_t)(min(wave * (BN / 4) + i * 8 + (ln >> 3), P.N - 1 - Q.c0) * kBytes);
        } else {
            colBase = (KIND == kDenseRowsGrad ? P.weights + (int64_t)Q.e * P.N * P.H * 2 : P.rows) + (int64_t)Q.c0 * 2;
#pragma unroll
            for (int s = 0; s < kSwC; ++s) {
                turnedC[s] = turned_piece(Const<BN>{}, s, P.H - Q.c0);
                if constexpr (KIND == kDenseRowsGrad) turnedC[s] += (lane / kLanesC) * ((uint32_t)P.H * 2);
                if constexpr (kTurnedR) fromC[s] = colBase + turnedC[s];
            }
        }
        if constexpr (kTurnedR) {
#pragma unroll
            for (int s = 0; s < kSwR; ++s) fromR[s] = P.dOut + (int64_t)Q.r0 * 2 + turned_piece(Const<BM>{}, s, P.N - Q.r0);
        }
        b += gridDim.x;
        next = find(b);
        if constexpr (KIND != kDenseWeightsGrad) fetch_entry(next);
    };
    // What the requests of step kq of tile Q need.  A step is one of its tile's, or (of a tile that does not exist) 0 or 1:
    // the weights' gradient's, of 64 entries each, go up to 2^25.
    auto advance = [&] {
        const int32_t k = uniform(kq);
        if constexpr (KIND != kDenseWeightsGrad) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                placeR[i] = P.rows + min(k * 128 + (piece ^ i * 64), kBytes - 16);
                placeC[i] = (uint32_t)min(k * 128 + (piece ^ i * 64), kBytes - 16);
            }
        }
        if constexpr (KIND == kDenseProduct) stepBase = uniform_pointer(colBase);
        if constexpr (KIND == kDenseRowsGrad) stepBase = uniform_pointer(colBase + (int64_t)(k * 64 + wave * 16) * ((uint32_t)P.H * 2));
        if constexpr (KIND == kDenseWeightsGrad) {
            const int32_t at = k * 64 + lane;
            const int32_t r = P.outRow ? listR : Q.lo + at, c = P.entryRow ? listC : Q.lo + at;
            const bool in = Q.e >= 0 && at < Q.hi - Q.lo && (uint32_t)r < (uint32_t)P.numOutRows && (uint32_t)c < (uint32_t)P.numRows;
            dead = ~__ballot(in);
            idxR = in ? r : 0;
            idxC = in ? c : 0;
        }
    };
    // The lists of the steps behind it, once all waves' requests of before have arrived.
    auto advance_lists = [&] {
        if constexpr (KIND == kDenseWeightsGrad) {
            if (kq + 2 < stepsQ)
                request_lists(Q, kq + 2, slot + 2);
            else
                request_lists(next, kq + 2 - stepsQ, slot + 2);
            read_lists(slot + 1);
            ++slot;
        }
    };
    // Gathered: the place of load t of the wave's LR + LC.
    auto prepare = [&](auto t) {
        constexpr int T = decltype(t)::value, I = T < LR ? T : T - LR, kPer = T < LR ? kPerR : kPerC, BX = T < LR ? BM : BN;
        constexpr int S = BX == 256 ? (I & 1) | (I >> 2) << 1 : 0;
        const uint32_t r = (uint32_t)__builtin_amdgcn_ds_bpermute((wave * 16 + lane / (64 / kPer) + I * kPer) * 4, T < LR ? idxR : idxC);
        src[T] = (T < LR ? fromR[S] : fromC[S]) + (uint64_t)r * (uint32_t)((T < LR ? P.N : P.H) * 2);
    };
    auto prepare_dead = [&] {  // of entries that are none, and behind the group's last: zeros
        if (!rarely(dead != 0)) return;
        const int ln = fresh();
#pragma unroll
        for (int t = 0; t < LR + LC; ++t) {
            const int kPer = t < LR ? kPerR : kPerC, i = t < LR ? t : t - LR;
            if (dead >> (wave * 16 + ln / (64 / kPer) + i * kPer) & 1) src[t] = zero;
        }
    };
    // Load t of the wave's LR + LC of the step (rows, then columns), into its part of a place in LDS.
    const uint32_t ringAt = lds_address(ring) + wave * (kPlace / 4);
    auto request = [&](auto t, uint32_t place) {
        constexpr int T = decltype(t)::value, I = T < LR ? T : T - LR;
        const uint32_t to = ringAt + place;
        if constexpr (KIND == kDenseWeightsGrad) {
            load_lds16_unseen<I * 1024>(src[T], to);
        } else if constexpr (T < LR) {
            load_lds16_unseen<I * 1024>(placeR[I & 1] + (uint64_t)rowi[I] * (uint32_t)kBytes, to);
        } else if constexpr (KIND == kDenseProduct) {
            load_lds16_unseen<I * 1024>(stepBase, colo[I] + placeC[I & 1], to);
        } else {
            constexpr int S = BN == 256 ? (I & 1) | (I >> 2) << 1 : 0;
            const int32_t left = P.N - 1 - uniform(kq) * 64 - wave * 16 - I * kPerC;  // rows behind the load's first
            if (!rarely(left < kPerC - 1))
                load_lds16_unseen<I * 1024>(uniform_pointer(stepBase + (int64_t)(I * kPerC) * ((uint32_t)P.H * 2)), turnedC[S], to);
            else  // the last row, where this lane's is behind it
                load_lds16_unseen<I * 1024>(stepBase + ((int64_t)(I * kPerC) + min(left - lane / kLanesC, 0)) * ((uint32_t)P.H * 2) + turnedC[S], to);
        }
    };
    // A step that has arrived, with places behind the end of the summed index (step k of its tile): zeros there, on
    // both sides, so that no value that is not part of the sum is multiplied.  (The weights' gradient loads them.)
    auto clear_tail = [&](int32_t k, uint32_t at) {
        if constexpr (KIND == kDenseWeightsGrad) return;
        if (!rarely((k + 1) * 128 > kBytes)) return;
        const u32x4 none = {0, 0, 0, 0};
        const int ln = fresh(), pc = ((ln & 7) ^ (ln >> 4)) * 16;
        uint8_t *const rb = ring + at, *const cb = rb + kPlace;
#pragma unroll
        for (int i = 0; i < LR; ++i)
            if (k * 128 + (pc ^ (i & 1) * 64) >= kBytes) *reinterpret_cast<u32x4 *>(rb + wave * (BM / 4) * 128 + i * 1024 + ln * 16) = none;
#pragma unroll
        for (int i = 0; i < LC; ++i) {
            const bool behind = kTurnedC ? k * 64 + wave * 16 + i * kPerC + ln / kLanesC >= P.N : k * 128 + (pc ^ (i & 1) * 64) >= kBytes;
            if (behind) *reinterpret_cast<u32x4 *>(cb + wave * (BN / 4) * 128 + i * 1024 + ln * 16) = none;
        }
        __syncthreads();
    };

    // ---- operands
    struct Half {
        u32x4 r[FR][2], c[FC][2];
    };
    const int l31 = lane & 31, far = lane >> 5, q = lane >> 4, j = lane & 15;
    // Rows along the summed index: the lane's row in a fragment -- rows in order; columns so that a lane's 16 sums are
    // two runs of eight: the instruction's row r is column r with bits 2 and 3 exchanged -- and the piece of 16 bytes.
    const int colOf = (l31 & 0x13) | (l31 >> 2 & 1) << 3 | (l31 >> 3 & 1) << 2;
    const int alongR = (wr + l31) * 128 + (far ^ (l31 >> 1 & 7)) * 16, alongC = (wc + colOf) * 128 + (far ^ (colOf >> 1 & 7)) * 16;
    // Turned: rows 8 (q / 2) + j / 4 (+ 4) of 16, columns 16 (q % 2) + 4 (j % 4) .. + 3 of 32 (with the same exchange).
    const int turnRowC = (8 * (q >> 1) + (j >> 2)) * (BN * 2) + (q & 1) * 32 + ((j & 1) * 8 + (j >> 1 & 1) * 4) * 2;
    const int turnRowR = (8 * (q >> 1) + (j >> 2)) * (BM * 2) + (q & 1) * 32 + (j & 3) * 8;
    const int swC = BN == 256 ? (j >> 2) | (q >> 1) << 2 : j >> 2, swR = BM == 256 ? (j >> 2) | (q >> 1) << 2 : j >> 2;
    int turnC[kTurnedC ? FC : 1], turnR[kTurnedR ? FR : 1];
    if constexpr (kTurnedC) {
#pragma unroll
        for (int f = 0; f < FC; ++f) turnC[f] = turnRowC + ((wc / 32 + f) ^ swC) * 64;
    }
    if constexpr (kTurnedR) {
#pragma unroll
        for (int f = 0; f < FR; ++f) turnR[f] = turnRowR + ((2 * f + (wave & 1)) ^ swR) * 64;
    }
    // The LDS reads of fragment F, chunk CH (32 bytes of the summed index) of half `half` of a step.
    auto read_r = [&](auto f, auto ch, Half &h, const uint8_t *rb, int half) {
        constexpr int F = decltype(f)::value, CH = decltype(ch)::value;
        if constexpr (kTurnedR) {
            const u32x2 lo = read_turned(rb + turnR[F] + (half * 32 + CH * 16) * (BM * 2));
            const u32x2 hi = read_turned(rb + turnR[F] + (half * 32 + CH * 16 + 4) * (BM * 2));
            h.r[F][CH] = u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {
            h.r[F][CH] = *reinterpret_cast<const u32x4 *>(rb + (alongR ^ (half * 64 + CH * 32)) + F * 8192);
        }
    };
    auto read_c = [&](auto f, auto ch, Half &h, const uint8_t *cb, int half) {
        constexpr int F = decltype(f)::value, CH = decltype(ch)::value;
        if constexpr (kTurnedC) {
            const u32x2 lo = read_turned(cb + turnC[F] + (half * 32 + CH * 16) * (BN * 2));
            const u32x2 hi = read_turned(cb + turnC[F] + (half * 32 + CH * 16 + 4) * (BN * 2));
            h.c[F][CH] = u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {
            h.c[F][CH] = *reinterpret_cast<const u32x4 *>(cb + (alongC ^ (half * 64 + CH * 32)) + F * 4096);
        }
    };
    // This wave's LDS reads are in its registers and all but its last `left` loads and stores are done; then all waves' are.
    auto meet = [&](auto left) {
        constexpr int L = decltype(left)::value;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((L & 15) | (L >> 4) << 14 | 0x70);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // The same where the results of `n` fragments of rows were stored since.
    auto meet_behind = [&](int32_t n) {
        constexpr int kPer = FC * 2 * (OUT32 ? 2 : 1);  // stores of a wave and fragment of rows
        each<FR + 1>([&](auto f) {
            constexpr int L = decltype(f)::value * kPer < 63 ? decltype(f)::value * kPer : 63;
            if (n == decltype(f)::value) __builtin_amdgcn_s_waitcnt((L & 15) | (L >> 4) << 14 | 0x70);
        });
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // LDS read n of a half, in the order in which the products need them.
    constexpr int kReads = 2 * (FR + FC);
    auto read = [&](auto n, Half &h, const uint8_t *rb, const uint8_t *cb, int half) {
        constexpr int CH = decltype(n)::value / (FR + FC), M = decltype(n)::value % (FR + FC);
        if constexpr (M == 0)
            read_r(Const<0>{}, Const<CH>{}, h, rb, half);
        else if constexpr (M <= FC)
            read_c(Const<M - 1>{}, Const<CH>{}, h, cb, half);
        else
            read_r(Const<M - FC>{}, Const<CH>{}, h, rb, half);
    };
    // The products of a half, one matrix instruction after the other, NJ fragments of rows of them; between(n, of) is
    // what goes behind product n of `of`, where the matrix instructions leave issue slots.
    auto multiply = [&](auto nj, auto first, const Half &h, auto &&between) {
        constexpr int NJ = decltype(nj)::value;
        hold_sums<FC * FR>();
        each<2 * NJ * FC>([&](auto n) {
            constexpr int Nn = decltype(n)::value, CH = Nn / (NJ * FC), J = Nn % (NJ * FC) / FC, I = Nn % FC;
            mfma_sums<I * FR + J, decltype(first)::value && CH == 0, INT8>(h.c[I][CH], h.r[J][CH]);
            between(Const<Nn>{}, Const<2 * NJ * FC>{});
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    if constexpr (KIND == kDenseWeightsGrad) {
        request_lists(next, 0, 0);
        request_lists(next, 1, 1);
        meet(Const<0>{});
        read_lists(0);
    } else {
        fetch_entry(next);
    }
    uint32_t at = 0;  // the places of step k: rows at `at`, columns behind them; of step k + 1 at at ^ kNext
    constexpr uint32_t kNext = 2 * kPlace;
    auto request_step = [&](uint32_t to) {
        advance();
        if constexpr (KIND == kDenseWeightsGrad) {
            each<LR + LC>([&](auto t) { prepare(t); });
            prepare_dead();
        }
        advance_lists();
        each<LR + LC>([&](auto t) { request(t, to + (decltype(t)::value < LR ? 0 : kPlace)); });
        ++kq;
        meet(Const<0>{});
    };
    turn_to_next();
    request_step(0);
    request_step(kNext);
    DenseTile T = Q;  // the tile that is computed, step k of `steps`
    int32_t k = 0, steps = stepsQ;
    clear_tail(0, 0);
    auto rows_of = [&](const DenseTile &t) { return KIND == kDenseWeightsGrad ? min(P.N - t.r0, BM) : t.hi - t.lo; };
    int32_t mine = ceil_div(rows_of(T), 64);  // fragments of rows of a wave
    int32_t stored = 0;                       // of the tile before, whose results are on their way
    Half h0, h1;
    each<kReads>([&](auto n) { read(n, h0, ring, ring + kPlace, 0); });

    auto step = [&](auto nj, auto first) {
        constexpr bool FIRST = decltype(first)::value;
        advance();
        const uint8_t *const rb = ring + at, *const cb = rb + kPlace, *const ro = ring + (at ^ kNext), *const co = ro + kPlace;
        constexpr int kLoads = LR + LC;
        multiply(nj, first, h0, [&](auto n, auto of) {
            constexpr int Nn = decltype(n)::value, kOf = decltype(of)::value;
            constexpr int kFirst = Nn * kReads / kOf, kEnd = (Nn + 1) * kReads / kOf;
            each<kEnd - kFirst>([&](auto m) { read(Const<kFirst + decltype(m)::value>{}, h1, rb, cb, 1); });
            if constexpr (KIND == kDenseWeightsGrad) {
                constexpr int kFirstP = Nn * kLoads / kOf, kEndP = (Nn + 1) * kLoads / kOf;
                each<kEndP - kFirstP>([&](auto m) { prepare(Const<kFirstP + decltype(m)::value>{}); });
            }
        });
        if constexpr (FIRST)
            meet_behind(stored);  // step 1 was there before the results' stores
        else
            meet(Const<0>{});
        clear_tail(k + 1 == steps ? 0 : k + 1, at ^ kNext);
        if constexpr (KIND == kDenseWeightsGrad) prepare_dead();
        advance_lists();
        multiply(nj, Const<0>{}, h1, [&](auto n, auto of) {
            constexpr int Nn = decltype(n)::value, kOf = decltype(of)::value;
            constexpr int kFirst = Nn * kReads / kOf, kEnd = (Nn + 1) * kReads / kOf;
            each<kEnd - kFirst>([&](auto m) { read(Const<kFirst + decltype(m)::value>{}, h0, ro, co, 0); });
            constexpr int kFirstQ = Nn * kLoads / kOf, kEndQ = (Nn + 1) * kLoads / kOf;
            each<kEndQ - kFirstQ>([&](auto m) {
                constexpr int M = kFirstQ + decltype(m)::value;
                request(Const<M>{}, at + (M < LR ? 0 : kPlace));
            });
        });
        ++kq, ++k;
        at ^= kNext;
    };
    // Stores a tile's results and begins the next; false where there is none.
    auto finish = [&] {
        mfma_done();
        uint8_t *base;
        if constexpr (KIND == kDenseWeightsGrad)
            base = P.out + ((int64_t)T.e * P.N + T.r0) * rowOut;
        else
            base = P.out + (int64_t)T.lo * rowOut;
        const int32_t bytes = rows_of(T) * rowOut;
        // a buffer that ends with the tile's last row; columns past the end are sent beyond it
        const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(base, 0, bytes, 0x00020000);
        const __amdgpu_buffer_rsrc_t add = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t *>(KIND == kDenseWeightsGrad && P.base ? P.base + (base - P.out) : base), 0, bytes, 0x00020000);
        const int ln = fresh(), low = ln & 31, high = ln >> 5;
        // Where a lane stores: rows low % 16 and 16 behind, 16 bytes; a row's four lanes hold 64 bytes that follow one
        // another (lanes that each stored their own sums would write 32 at a time: a tenth slower at the weights' gradient
        // of 333 entries, 16 experts of 1024 x 1000, fp32).
        constexpr int kRuns = OUT32 ? 2 : 1;  // of 64 bytes in a fragment's row
        const int32_t outside = 0x7ffffff0, mineC = T.c0 + wc + high * (OUT32 ? 4 : 8) + (low >> 4) * (OUT32 ? 8 : 16);
        int32_t at[FC][kRuns];
        float cs[FC][2][8];
#pragma unroll
        for (int i = 0; i < FC; ++i) {
#pragma unroll
            for (int p = 0; p < kRuns; ++p) {
                const int32_t c = mineC + i * 32 + p * 16;
                at[i][p] = c < C ? (wr + (low & 15)) * rowOut + c * (OUT32 ? 4 : 2) : outside;
            }
            if constexpr (INT8) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const int32_t c = T.c0 + wc + i * 32 + p * 16 + high * 8;
                    const float *s = P.weightScales + (int64_t)T.e * P.N;
                    const f32x4_dword lo = *reinterpret_cast<const f32x4_dword *>(s + min(c, P.N - 4));
                    const f32x4_dword hi = *reinterpret_cast<const f32x4_dword *>(s + min(c + 4, P.N - 4));
#pragma unroll
                    for (int v = 0; v < 4; ++v) cs[i][p][v] = lo[v], cs[i][p][4 + v] = hi[v];
                }
            }
        }
        each<FR>([&](auto f) {
            constexpr int F = decltype(f)::value;
            if (F >= mine) return;
            const uint32_t down = (uint32_t)(F * 64) * (uint32_t)rowOut;
            RowInfo info{};
            if constexpr (KIND != kDenseWeightsGrad) info = rowInfo[(turns & 1) ^ 1][wr + F * 64 + low];
            // What the gradient is added to, of all the fragment's columns at once: so many loads are under way together.
            constexpr int kAdd = KIND == kDenseWeightsGrad ? FC : 1, kAddRuns = OUT32 ? 2 : 1;
            u32x4 before[kAdd][2][kAddRuns];
            if (KIND == kDenseWeightsGrad && P.base) {
#pragma unroll
                for (int i = 0; i < kAdd; ++i)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const int32_t c = T.c0 + wc + i * 32 + p * 16 + high * 8;
                        const int32_t from = (int32_t)((wr + low) * rowOut + c * (OUT32 ? 4 : 2) + down);
#pragma unroll
                        for (int q = 0; q < kAddRuns; ++q)
                            before[i][p][q] = __builtin_amdgcn_raw_buffer_load_b128(add, c < C ? from + q * 16 : outside, 0, 0);
                    }
            }
            each<FC>([&](auto ii) {
                constexpr int i = decltype(ii)::value;
                // v[p]: columns 16 p + 8 high .. + 7 of row `low`
                float v[2][8];
                each<16>([&](auto x) {
                    constexpr int X = decltype(x)::value;
                    if constexpr (X % 8 == 0) hold_sums<FC * FR>();
                    const uint32_t sum = read_sum<i * FR + F, X>();
                    if constexpr (INT8)
                        v[X / 8][X % 8] = (float)(int32_t)sum * info.scale * cs[i][X / 8][X % 8];
                    else
                        v[X / 8][X % 8] = __uint_as_float(sum);
                });
                if constexpr (KIND != kDenseWeightsGrad) {
#pragma unroll
                    for (int x = 0; x < 16; ++x) v[x / 8][x % 8] = info.there ? v[x / 8][x % 8] * info.factor : 0.0f;
                } else if (P.base) {
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const u32x4(&a)[kAddRuns] = before[i % kAdd][p];
                        if constexpr (OUT32) {
#pragma unroll
                            for (int x = 0; x < 8; ++x) v[p][x] += __uint_as_float(a[x / 4 % kAddRuns][x % 4]);
                        } else {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                v[p][2 * x] += __uint_as_float(a[0][x] << 16), v[p][2 * x + 1] += __uint_as_float(a[0][x] & 0xffff0000u);
                        }
                    }
                }
#pragma unroll
                for (int p = 0; p < kRuns; ++p) {
                    u32x4 a, b;  // the two that trade lanes: fp32's halves of a run, bf16's two runs
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t lo, hi;
                        if constexpr (OUT32) {
                            lo = __float_as_uint(v[p][x]), hi = __float_as_uint(v[p][4 + x]);
                            swap32(lo, hi);
                        } else {
                            lo = bf16_pair(v[0][2 * x], v[0][2 * x + 1]), hi = bf16_pair(v[1][2 * x], v[1][2 * x + 1]);
                        }
                        swap16(lo, hi);
                        a[x] = lo;
                        b[x] = hi;
                    }
                    const uint32_t to = (uint32_t)at[i][p] + down;
                    __builtin_amdgcn_raw_buffer_store_b128(a, out, (int)to, 0, 0);
                    __builtin_amdgcn_raw_buffer_store_b128(b, out, (int)(to + 16u * (uint32_t)rowOut), 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        });
        hold_sums<FC * FR>();
        stored = mine;
        T = Q;
        k = 0;
        steps = stepsQ;
        mine = ceil_div(rows_of(T), 64);
        return T.e >= 0;
    };
    // f(fragments of rows that a wave has in this tile), a constant
    auto with_fragments = [&](auto &&f) {
        if constexpr (FR == 4) {
            if (mine > 3) return f(Const<4>{});
            if (mine == 3) return f(Const<3>{});
        }
        if (mine > 1) return f(Const<2>{});
        f(Const<1>{});
    };
    for (bool turned = false;;) {
        if (!turned && k + 2 >= steps) {  // the last two steps request the next tile's first two
            turn_to_next();
            turned = true;
        }
        if (k == 0) with_fragments([&](auto nj) { step(nj, Const<1>{}); });
        const int32_t until = turned ? steps : steps - 2;
        with_fragments([&](auto nj) {
            while (k < until) step(nj, Const<0>{});
        });
        if (k < steps) continue;
        if (!finish()) break;
        turned = false;
    }
    __builtin_amdgcn_s_waitcnt(0x0f70);  // nothing of this wave is on its way into LDS when it ends
}

template <DenseKind KIND, bool INT8, int BM, int BN>
hipError_t launch_tiles(const DenseParams &P, bool out32, hipStream_t stream) {
    int64_t tiles;
    if (KIND == kDenseWeightsGrad)
        tiles = (int64_t)P.E * ceil_div(P.N, BM) * ceil_div(P.H, BN);
    else  // row tiles at most: one partly filled for each expert
        tiles = ((int64_t)P.maxEntries / BM + (P.E < P.maxEntries ? P.E : P.maxEntries)) * ceil_div(KIND == kDenseProduct ? P.N : P.H, BN);
    if (tiles > INT32_MAX / 2) return hipErrorInvalidConfiguration;
    int device = 0, cus = 0;
    hipError_t err = hipGetDevice(&device);
    if (err == hipSuccess) err = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device);
    if (err != hipSuccess) return err;
    // as many blocks as run at once, a multiple of the 8 XCDs
    const int64_t most = (int64_t)ceil_div(cus * (BM * BN > 128 * 128 ? 1 : 2), 8) * 8, blocks = (tiles + 7) / 8 * 8;
    const dim3 grid((uint32_t)(blocks < most ? blocks : most));
    if (out32)
        hipLaunchKernelGGL((dense_tile_kernel<KIND, INT8, BM, BN, true>), grid, dim3(256), 0, stream, P);
    else
        hipLaunchKernelGGL((dense_tile_kernel<KIND, INT8, BM, BN, false>), grid, dim3(256), 0, stream, P);
    return hipGetLastError();
}

}  // namespace
}  // namespace epdc
