// The products of bf16 and int8 rows with the experts' weights, and the bf16
// product's two gradients, for gfx950: over a group's entries i
//   product           out[i][n]   = sum_h rows[r_i][h] W[n][h]
//   rows' gradient    dRows[i][h] = sum_n dOut[r_i][n] W[n][h]
//   weights' gradient dW[n][h]    = sum_i dOut[o_i][n] rows[r_i][h]
//
// Tiles of 256 x 256 or 128 x 128 of the output, through LDS, with
// v_mfma_f32_32x32x16_bf16 (v_mfma_i32_32x32x32_i8); plan_dense chooses.
#include "tiles.h"

namespace epdc {
namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_dword __attribute__((ext_vector_type(4), aligned(4)));  // 16 bytes at 4-byte alignment

// The sums of 32 x 32 products stay in accumulation registers that the matrix
// instruction updates in place, in the order written.  The compiler does not
// see the instruction: its operands must not come from a vector instruction
// just before it, and its sums are read behind mfma_done().
__device__ __forceinline__ void mfma_inplace(f32x16 &c, u32x4 a, u32x4 b) {
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma_inplace(i32x16 &c, u32x4 a, u32x4 b) {
    asm volatile("v_mfma_i32_32x32x32_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
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

// Where a tile of the output lies: expert, entries [lo, hi) of its group (of
// the tile, but for the weights' gradient), rows from r0, columns from c0.
struct DenseTile {
    int32_t e, lo, hi, r0, c0;
};

// A BM x BN tile of the output by four waves, (BM/2) x (BN/2) each, in 32 x 32
// fragments; the output's columns are the instruction's rows and its rows the
// instruction's columns, so a lane ends with runs of 8 consecutive columns of
// one row.
//
// The summed index goes in steps of 128 bytes of it (64 bf16, 128 int8) through
// two pairs of LDS buffers, loaded by the memory pipeline itself.  A step is
// two halves; the operands of a half are read into registers during the half
// before:
//     read half 1 of step k        | products of half 0
//     wait: step k+1 has arrived (requested one whole step ago); barrier
//     request step k+2 into step k's buffers
//     read half 0 of step k+1      | products of half 1
// The steps of a block's tiles follow one another without a gap: behind a
// tile's last step come the next tile's first (a stride of the grid further),
// requested while the last ones are computed; a tile's results are stored with
// them under way.  A tile has two steps at least (of zeros, if need be).
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
    using Acc = std::conditional_t<INT8, i32x16, f32x16>;
    constexpr bool kTurnedC = KIND != kDenseProduct, kTurnedR = KIND == kDenseWeightsGrad;
    constexpr int ES = INT8 ? 1 : 2;            // bytes of an element
    constexpr int FR = BM / 64, FC = BN / 64;   // fragments of a wave
    constexpr int LR = BM / 32, LC = BN / 32;   // LDS loads of a wave per step (1 KB each)
    __shared__ __attribute__((aligned(16))) uint8_t rbuf0[BM * 128], rbuf1[BM * 128], cbuf0[BN * 128], cbuf1[BN * 128];
    // The weights' gradient: rows of a step's entries (of dOut, of rows), of four steps that follow one another.
    __shared__ int32_t list[4][2][64];
    const int32_t C = KIND == kDenseProduct ? P.N : P.H;  // the output's columns
    const int32_t RT = ceil_div(P.N, BM), CT = ceil_div(C, BN);
    const int32_t rowOut = C * (OUT32 ? 4 : 2);
    const int32_t kBytes = KIND == kDenseProduct ? P.H * ES : P.N * ES;  // of a row of the summed index (not the weights' gradient)
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wr = (wave & 1) * (BM / 2), wc = (wave >> 1) * (BN / 2);
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
            const TileAt a = find_tile<BM, BN>(P, groups, CT, b);
            t = DenseTile{a.e, a.m0, a.hi, a.m0, a.n0};
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
    // Rows along the summed index: where this lane's rows begin in the rows' array, their offsets from the tile's first
    // column, and the place in a row (of even and odd loads) that it requests.
    const uint8_t *rowp[kTurnedR ? 1 : LR];
    uint32_t colo[kTurnedC ? 1 : LC];
    const int piece = ((lane & 7) ^ (lane >> 4)) * 16;  // of a step, in even loads (in odd ones ^ 64)
    uint32_t place[2] = {0, 0};
    const uint8_t *stepBase = nullptr;  // columns that are not gathered: from where this step's are requested
    int32_t entryRow = -1;  // the row of entry wave * (BM/4) + lane of the next tile, on its way
    // Turned rows: lanes of a row of BX elements, rows of a load, and the 16-byte piece that this lane requests.
    constexpr int kLanesR = BM / 8, kPerR = 64 / kLanesR, kLanesC = BN / 8, kPerC = 64 / kLanesC;
    uint32_t turnedR[kTurnedR ? (BM == 256 ? 4 : 1) : 1], turnedC[kTurnedC ? (BN == 256 ? 4 : 1) : 1];
    // offset of the piece in the tile's part of a row, by the load's swizzle; behind the row's end the last piece
    auto turned_piece = [&](auto bx, int s, int32_t left) {
        constexpr int BX = decltype(bx)::value;
        const int p = lane & (BX / 8 - 1);
        const int sw = BX == 256 ? ((s & 1) * 2 + (lane >> 5)) | (s >> 1) << 2 : lane >> 4;
        return (uint32_t)min((p ^ (sw << 2)) * 16, left * 2 - 16);
    };
    int32_t listR = 0, listC = 0;  // the weights' gradient: rows of entry wave * 16 + lane % 16 of the next step, as listed
    int32_t idxR = -1, idxC = -1;  // and of the step that is requested; -1: none
    uint32_t slot = 0;             // of that step among all, % 4 its lists' place
    const uint8_t *colBase = nullptr, *rowBase = nullptr;
    auto fetch_entry = [&](const DenseTile &t) {  // product, rows' gradient
        const int32_t ent = t.lo + wave * (BM / 4) + (lane & (BM / 4 - 1));
        entryRow = -1;
        if (t.e >= 0 && ent < t.hi) entryRow = P.entryRow ? P.entryRow[ent] : ent;
    };
    // Weights' gradient: the lists of step k of a tile, on their way into a place; wave 0 asks for dOut's, wave 1 for rows'.
    auto request_lists = [&](const DenseTile &t, int32_t k, uint32_t place) {
        const int32_t *from = wave == 0 ? P.outRow : P.entryRow;
        if (wave >= 2 || !from || t.e < 0) return;
        const int32_t at = k * 64 + lane;
        if (at < t.hi - t.lo) load_lds4_unseen(from + t.lo + at, lds_address(list[place & 3][wave]));
    };
    auto read_lists = [&](uint32_t place) {
        if (P.outRow) listR = list[place & 3][0][wave * 16 + (lane & 15)];
        if (P.entryRow) listC = list[place & 3][1][wave * 16 + (lane & 15)];
    };
    // Tile Q becomes `next`, or stays where there is none: what is requested then is not used.
    auto turn_to_next = [&] {
        kq = 0;
        if (next.e < 0) {
            Q.e = -1;
            stepsQ = INT32_MAX;
            return;
        }
        Q = next;
        stepsQ = steps_of(Q);
        if constexpr (KIND != kDenseWeightsGrad) {
            const int32_t row = (uint32_t)entryRow < (uint32_t)P.numRows ? entryRow : 0;  // an entry without a row: any row, and zeros stored
#pragma unroll
            for (int i = 0; i < LR; ++i) rowp[i] = P.rows + (int64_t)__shfl(row, i * 8 + (lane >> 3)) * kBytes;
        }
        if constexpr (KIND == kDenseProduct) {
            colBase = P.weights + ((int64_t)Q.e * P.N + Q.c0) * kBytes;
#pragma unroll
            for (int i = 0; i < LC; ++i) colo[i] = (uint32_t)(min(wave * (BN / 4) + i * 8 + (lane >> 3), P.N - 1 - Q.c0) * kBytes);
        } else {
            colBase = (KIND == kDenseRowsGrad ? P.weights + (int64_t)Q.e * P.N * P.H * 2 : P.rows) + (int64_t)Q.c0 * 2;
#pragma unroll
            for (int s = 0; s < (BN == 256 ? 4 : 1); ++s) {
                turnedC[s] = turned_piece(Const<BN>{}, s, P.H - Q.c0);
                if constexpr (KIND == kDenseRowsGrad) turnedC[s] += (lane / kLanesC) * ((uint32_t)P.H * 2);
            }
            if constexpr (kTurnedR) {
                rowBase = P.dOut + (int64_t)Q.r0 * 2;
#pragma unroll
                for (int s = 0; s < (BM == 256 ? 4 : 1); ++s) turnedR[s] = turned_piece(Const<BM>{}, s, P.N - Q.r0);
            }
        }
        b += gridDim.x;
        next = find(b);
        if constexpr (KIND != kDenseWeightsGrad) fetch_entry(next);
    };
    // Step kq of tile Q, or the first of the next: what its requests need.
    auto advance = [&] {
        if (kq == stepsQ) turn_to_next();
        const int32_t k = uniform(kq);
        if constexpr (KIND != kDenseWeightsGrad) {
#pragma unroll
            for (int i = 0; i < 2; ++i) place[i] = (uint32_t)min(min(k, 1 << 22) * 128 + (piece ^ i * 64), kBytes - 16);
        }
        if constexpr (KIND == kDenseProduct) stepBase = uniform_pointer(colBase);
        if constexpr (KIND == kDenseRowsGrad) stepBase = uniform_pointer(colBase + (int64_t)(min(k, 1 << 22) * 64 + wave * 16) * ((uint32_t)P.H * 2));
        if constexpr (KIND == kDenseWeightsGrad) {
            const int32_t at = k * 64 + wave * 16 + (lane & 15);
            const int32_t r = P.outRow ? listR : Q.lo + at, c = P.entryRow ? listC : Q.lo + at;
            const bool in = Q.e >= 0 && at < Q.hi - Q.lo && (uint32_t)r < (uint32_t)P.numOutRows && (uint32_t)c < (uint32_t)P.numRows;
            idxR = in ? r : -1;
            idxC = in ? c : -1;
            if (k + 2 < stepsQ)
                request_lists(Q, k + 2, slot + 2);
            else
                request_lists(next, k + 2 - stepsQ, slot + 2);
            read_lists(slot + 1);
            ++slot;
        }
    };
    // The row's index of a turned load's lanes, from the lanes that hold them.
    auto spread = [&](auto per, int32_t idx, int i) {
        constexpr int kPer = decltype(per)::value;
        int32_t v = __builtin_amdgcn_readlane(idx, i * kPer);
#pragma unroll
        for (int q = 1; q < kPer; ++q) v = lane / (64 / kPer) == q ? __builtin_amdgcn_readlane(idx, i * kPer + q) : v;
        return v;
    };
    // Load t of the wave's LR + LC of the step, into its places in LDS from rb and cb.
    const uint32_t rto0 = lds_address(rbuf0 + wave * (BM / 4) * 128), rto1 = lds_address(rbuf1 + wave * (BM / 4) * 128);
    const uint32_t cto0 = lds_address(cbuf0 + wave * (BN / 4) * 128), cto1 = lds_address(cbuf1 + wave * (BN / 4) * 128);
    auto request = [&](auto t, uint32_t rb, uint32_t cb) {
        constexpr int T = decltype(t)::value, I = T < LR ? T : T - LR, BX = T < LR ? BM : BN, S = BX == 256 ? (I & 1) | (I >> 2) << 1 : 0;
        if constexpr (KIND == kDenseWeightsGrad) {
            const int32_t r = T < LR ? spread(Const<kPerR>{}, idxR, I) : spread(Const<kPerC>{}, idxC, I);
            const uint8_t *from = T < LR ? rowBase : colBase;
            const uint64_t off = (uint64_t)(uint32_t)r * ((uint32_t)(T < LR ? P.N : P.H) * 2) + (T < LR ? turnedR[S] : turnedC[S]);
            load_lds16_unseen<I * 1024>(r < 0 ? zero : from + off, T < LR ? rb : cb);
        } else if constexpr (T < LR) {
            load_lds16_unseen<I * 1024>(rowp[I] + place[I & 1], rb);
        } else if constexpr (KIND == kDenseProduct) {
            load_lds16_unseen<I * 1024>(stepBase, colo[I] + place[I & 1], cb);
        } else {
            const int32_t left = P.N - 1 - uniform(kq) * 64 - wave * 16 - I * kPerC;  // rows behind the load's first
            if (left >= kPerC - 1)
                load_lds16_unseen<I * 1024>(uniform_pointer(stepBase + (int64_t)(I * kPerC) * ((uint32_t)P.H * 2)), turnedC[S], cb);
            else  // the last row, where this lane's is behind it
                load_lds16_unseen<I * 1024>(stepBase + ((int64_t)(I * kPerC) + min(left - lane / kLanesC, 0)) * ((uint32_t)P.H * 2) + turnedC[S], cb);
        }
    };
    // A step that has arrived, with places behind the end of the summed index (step k of its tile): zeros there, on
    // both sides, so that no value that is not part of the sum is multiplied.  (The weights' gradient loads them.)
    auto clear_tail = [&](int32_t k, uint8_t *rb, uint8_t *cb) {
        if constexpr (KIND == kDenseWeightsGrad) return;
        if ((k + 1) * 128 <= kBytes) return;
        const u32x4 none = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < LR; ++i)
            if (k * 128 + (piece ^ (i & 1) * 64) >= kBytes) *reinterpret_cast<u32x4 *>(rb + wave * (BM / 4) * 128 + i * 1024 + lane * 16) = none;
#pragma unroll
        for (int i = 0; i < LC; ++i) {
            const bool behind = kTurnedC ? k * 64 + wave * 16 + i * kPerC + lane / kLanesC >= P.N : k * 128 + (piece ^ (i & 1) * 64) >= kBytes;
            if (behind) *reinterpret_cast<u32x4 *>(cb + wave * (BN / 4) * 128 + i * 1024 + lane * 16) = none;
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
        for (int f = 0; f < FR; ++f) turnR[f] = turnRowR + ((wr / 32 + f) ^ swR) * 64;
    }
    constexpr int kReadsC = FC * 2 * (kTurnedC ? 2 : 1), kReadsR = FR * 2 * (kTurnedR ? 2 : 1), kReads = kReadsC + kReadsR;
    // LDS read n of half `half` of a step: those of the first 32 bytes of the summed index first.
    auto read = [&](auto n, Half &h, const uint8_t *rb, const uint8_t *cb, int half) {
        constexpr int Nn = decltype(n)::value, CH = Nn >= kReads / 2, M = Nn - CH * (kReads / 2);
        if constexpr (M < kReadsC / 2) {
            if constexpr (kTurnedC) {
                constexpr int F = M / 2, X = M % 2;
                const u32x2 v = read_turned(cb + turnC[F] + (half * 32 + CH * 16 + X * 4) * (BN * 2));
                h.c[F][CH][2 * X] = v.x;
                h.c[F][CH][2 * X + 1] = v.y;
            } else {
                h.c[M][CH] = *reinterpret_cast<const u32x4 *>(cb + (alongC ^ (half * 64 + CH * 32)) + M * 4096);
            }
        } else {
            constexpr int MR = M - kReadsC / 2;
            if constexpr (kTurnedR) {
                constexpr int F = MR / 2, X = MR % 2;
                const u32x2 v = read_turned(rb + turnR[F] + (half * 32 + CH * 16 + X * 4) * (BM * 2));
                h.r[F][CH][2 * X] = v.x;
                h.r[F][CH][2 * X + 1] = v.y;
            } else {
                h.r[MR][CH] = *reinterpret_cast<const u32x4 *>(rb + (alongR ^ (half * 64 + CH * 32)) + MR * 4096);
            }
        }
    };
    Acc acc[FC][FR];
    // The products of a half, one matrix instruction after the other; dealt out between them the reads of the next
    // half and, with REQUEST, the requests of step kq.
    auto multiply = [&](auto request_too, const Half &h, Half &nx, const uint8_t *rb, const uint8_t *cb, int half, uint32_t rq,
                        uint32_t cq) {
        constexpr bool REQUEST = decltype(request_too)::value;
        constexpr int kAll = 2 * FR * FC;
        each<kAll>([&](auto n) {
            constexpr int Nn = decltype(n)::value, CH = Nn / (FR * FC), J = Nn % (FR * FC) / FC, I = Nn % FC;
            mfma_inplace(acc[I][J], h.c[I][CH], h.r[J][CH]);
            constexpr int kFirst = Nn * kReads / kAll, kEnd = (Nn + 1) * kReads / kAll;
            each<kEnd - kFirst>([&](auto m) { read(Const<kFirst + decltype(m)::value>{}, nx, rb, cb, half); });
            if constexpr (REQUEST) {
                constexpr int kFirstQ = Nn * (LR + LC) / kAll, kEndQ = (Nn + 1) * (LR + LC) / kAll;
                each<kEndQ - kFirstQ>([&](auto m) { request(Const<kFirstQ + decltype(m)::value>{}, rq, cq); });
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // This wave's LDS reads are in its registers and all but its last `left` loads and stores are done; then all waves' are.
    auto meet = [&](auto left) {
        constexpr int L = decltype(left)::value;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((L & 15) | (L >> 4) << 14 | 0x70);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    auto clear = [&] {
#pragma unroll
        for (int i = 0; i < FC; ++i)
#pragma unroll
            for (int n = 0; n < FR; ++n) {
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][n][v] = 0;
                asm volatile("" : "+a"(acc[i][n]));
            }
    };

    if constexpr (KIND == kDenseWeightsGrad) {
        request_lists(next, 0, 0);
        request_lists(next, 1, 1);
        meet(Const<0>{});
        read_lists(0);
    } else {
        fetch_entry(next);
    }
    advance();
    each<LR + LC>([&](auto t) { request(t, rto0, cto0); });
    ++kq;
    advance();
    each<LR + LC>([&](auto t) { request(t, rto1, cto1); });
    ++kq;
    DenseTile T = Q;  // the tile that is computed, step k of `steps`
    int32_t k = 0, steps = stepsQ;
    clear();
    meet(Const<0>{});
    clear_tail(0, rbuf0, cbuf0);
    Half h0, h1;
    each<kReads>([&](auto n) { read(n, h0, rbuf0, cbuf0, 0); });

    // Of the tile's rows, as its last step begins: the entries' weights (and scales), and which have no row.
    float factor[FR];
    float scale[FR];
    int32_t rowOf[FR];
    // Stores of results per wave and tile, whatever the tile holds.
    constexpr int kStores = FC * FR * 2 * (OUT32 ? 2 : 1);
    auto step = [&](const uint8_t *rb, const uint8_t *cb, uint8_t *ro, uint8_t *co, uint32_t rto, uint32_t cto) {
        const bool last = k + 1 == steps;
        if constexpr (KIND != kDenseWeightsGrad) {
            if (last) {
#pragma unroll
                for (int n = 0; n < FR; ++n) {
                    const int32_t ent = min(T.lo + wr + n * 32 + l31, T.hi - 1);
                    rowOf[n] = P.entryRow ? P.entryRow[ent] : ent;
                    factor[n] = P.entryWeight ? P.entryWeight[ent] : 1.0f;
                }
            }
        }
        multiply(Const<0>{}, h0, h1, rb, cb, 1, rto, cto);
        if (k == 0)
            meet(Const<kStores < 63 ? kStores : 63>{});  // step 1 was there before the results' stores
        else
            meet(Const<0>{});
        if constexpr (KIND != kDenseWeightsGrad) {
            if (last) {
#pragma unroll
                for (int n = 0; n < FR; ++n) {  // for the compiler: they have arrived here
                    asm volatile("" : "+v"(rowOf[n]));
                    asm volatile("" : "+v"(factor[n]));
                }
            }
        }
        if constexpr (INT8) {
            if (last) {
#pragma unroll
                for (int n = 0; n < FR; ++n) {
                    scale[n] = 0.0f;
                    if ((uint32_t)rowOf[n] < (uint32_t)P.numRows) scale[n] = P.rowScales[rowOf[n]];
                }
            }
        }
        clear_tail(last ? 0 : k + 1, ro, co);
        advance();
        multiply(Const<1>{}, h1, h0, ro, co, 0, rto, cto);
        ++kq;
        ++k;
        return last;
    };
    // Stores a tile's results and begins the next; false where there is none.
    auto finish = [&] {
        mfma_done();
        uint8_t *base;
        int32_t rows;
        if constexpr (KIND == kDenseWeightsGrad) {
            base = P.out + ((int64_t)T.e * P.N + T.r0) * rowOut;
            rows = min(P.N - T.r0, BM);
        } else {
            base = P.out + (int64_t)T.lo * rowOut;
            rows = T.hi - T.lo;
        }
        // a buffer that ends with the tile's last row; columns past the end are sent beyond it
        const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(base, 0, rows * rowOut, 0x00020000);
        const __amdgpu_buffer_rsrc_t add = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t *>(KIND == kDenseWeightsGrad && P.base ? P.base + (base - P.out) : base), 0, rows * rowOut, 0x00020000);
#pragma unroll
        for (int i = 0; i < FC; ++i) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int32_t c = T.c0 + wc + i * 32 + p * 16 + far * 8;
                float cs[8];
                if constexpr (INT8) {
                    const float *s = P.weightScales + (int64_t)T.e * P.N;
                    const f32x4_dword lo = *reinterpret_cast<const f32x4_dword *>(s + min(c, P.N - 4));
                    const f32x4_dword hi = *reinterpret_cast<const f32x4_dword *>(s + min(c + 4, P.N - 4));
#pragma unroll
                    for (int v = 0; v < 4; ++v) cs[v] = lo[v], cs[4 + v] = hi[v];
                }
#pragma unroll
                for (int n = 0; n < FR; ++n) {
                    float v[8];
                    asm volatile("" : "+a"(acc[i][n]));  // not copied out before they are needed
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        v[x] = (float)acc[i][n][p * 8 + x];
                        if constexpr (INT8) v[x] = v[x] * scale[n] * cs[x];
                    }
                    const int32_t outside = 0x7ffffff0, at = (wr + n * 32 + l31) * rowOut + c * (OUT32 ? 4 : 2);
                    const int32_t at0 = c < C ? at : outside, at1 = c + 4 < C ? at + 16 : outside;
                    if constexpr (KIND != kDenseWeightsGrad) {
                        const bool none = (uint32_t)rowOf[n] >= (uint32_t)P.numRows;
#pragma unroll
                        for (int x = 0; x < 8; ++x) v[x] = none ? 0.0f : v[x] * factor[n];
                    } else if (P.base) {
                        const u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(add, at0, 0, 0);
                        if constexpr (OUT32) {
                            const u32x4 a1 = __builtin_amdgcn_raw_buffer_load_b128(add, at1, 0, 0);
#pragma unroll
                            for (int x = 0; x < 4; ++x) v[x] += __uint_as_float(a[x]), v[4 + x] += __uint_as_float(a1[x]);
                        } else {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                v[2 * x] += __uint_as_float(a[x] << 16), v[2 * x + 1] += __uint_as_float(a[x] & 0xffff0000u);
                        }
                    }
                    if constexpr (OUT32) {
                        __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                                                     __float_as_uint(v[3])}, out, at0, 0, 0);
                        __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                                                                     __float_as_uint(v[7])}, out, at1, 0, 0);
                    } else {
                        __builtin_amdgcn_raw_buffer_store_b128(
                            u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])}, out, at0, 0, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        T = Q;
        k = 0;
        steps = stepsQ;
        clear();
        return T.e >= 0;
    };
    for (;;) {
        if (step(rbuf0, cbuf0, rbuf1, cbuf1, rto0, cto0) && !finish()) break;
        if (step(rbuf1, cbuf1, rbuf0, cbuf0, rto1, cto1) && !finish()) break;
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

hipError_t launch_dense(const DenseParams &P, DenseKind kind, bool int8, bool out32, hipStream_t stream) {
    const bool large = plan_dense(kind, P.E, P.N, P.H, P.maxEntries) == kDenseTiles256;
    switch (kind) {
    case kDenseProduct:
        if (int8) return large ? launch_tiles<kDenseProduct, true, 256, 256>(P, out32, stream) : launch_tiles<kDenseProduct, true, 128, 128>(P, out32, stream);
        return large ? launch_tiles<kDenseProduct, false, 256, 256>(P, out32, stream) : launch_tiles<kDenseProduct, false, 128, 128>(P, out32, stream);
    case kDenseRowsGrad:
        return large ? launch_tiles<kDenseRowsGrad, false, 256, 256>(P, out32, stream) : launch_tiles<kDenseRowsGrad, false, 128, 128>(P, out32, stream);
    case kDenseWeightsGrad:
        return large ? launch_tiles<kDenseWeightsGrad, false, 256, 256>(P, out32, stream) : launch_tiles<kDenseWeightsGrad, false, 128, 128>(P, out32, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace epdc
