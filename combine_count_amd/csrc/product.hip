// The experts' product for gfx950: out[i] = w_i * rows[r_i] . weights[e]^T for
// every entry i of every expert e, fp4x2 rows and weights with block scales.
//
// v_mfma_scale_f32_16x16x128_f8f6f4: D[16][16] += A[16][128] B[128][16], each
// operand element times its 32-block's power-of-two scale, fp32 sums.  Lane l
// holds row (or column) l % 16, elements [32 (l/16), 32 (l/16) + 32) -- one
// block, 16 bytes -- and that block's scale byte; of the result column l % 16,
// rows 4 (l/16) .. + 3.
//
// Three kernels (plan_product chooses): 256x256 and 128x128 tiles through LDS
// where experts have many entries, bound by the matrix cores (32768 entries of
// 32 experts, 4096 x 7168: 0.55 ms, 3.5 PFLOP/s; a loop of the instruction
// alone reaches 6.7), and weights streamed into registers where they have few,
// bound by the memory (64 entries: 83 us, 5.2 TB/s).
#include "ops_internal.h"

namespace epdc {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kFp4 = 4;  // the instruction's operand format

// SA, SB: which byte of sa, sb holds the lane's scale.
template <int SA, int SB>
__device__ __forceinline__ f32x4 mfma_fp4(u32x4 a, u32x4 b, f32x4 c, int32_t sa, int32_t sb) {
    const i32x8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const i32x8 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, kFp4, kFp4, SA, sa, SB, sb);
}

// The same, the sums in accumulation registers that it updates in place, and in
// the order written (the compiler's own allocation of 64 such sums moved them
// between register files inside the loop).  The compiler does not see the
// matrix instruction: its operands must not come from a vector instruction
// just before it, and its results are read behind mfma_done().
template <int SA, int SB>
__device__ __forceinline__ void mfma_fp4_inplace(f32x4 &c, u32x4 a, u32x4 b, int32_t sa, int32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%6,0] op_sel_hi:[%7,%8,0] cbsz:4 blgp:4"
                 : "+a"(c)
                 : "v"(a), "v"(b), "v"(sa), "v"(sb), "n"(SA & 1), "n"(SB & 1), "n"(SA >> 1), "n"(SB >> 1));
}
__device__ __forceinline__ void mfma_done() { asm volatile("s_nop 15\n\ts_nop 15"); }

// Two values as bf16, the first low, rounded to nearest even.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

typedef uint32_t u32x2_dword __attribute__((ext_vector_type(2), aligned(4)));  // 8 bytes at 4-byte alignment

// 16 bytes per lane from memory into LDS at lds + lane * 16 (lds the same in
// all lanes), counted by vmcnt: from rs' base at voff (per lane) + soff.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t rs, uint32_t voff, int32_t soff, uint8_t *lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void *)lds, 16, (int)voff, soff, 0, 0);
}
__device__ __forceinline__ void load_lds16(const uint8_t *src, uint8_t *lds) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                     (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t *base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, 0xffffffff, 0x00020000);
}

// What goes between the products of a half besides the reads of the next.
constexpr int kRequest = 1, kTurn = 2;

// Where a block's tile lies: expert, entries [m0, hi), columns from n0.
struct TileAt {
    int32_t e, m0, hi, n0;
};

// The groups as a wave holds them, 64 experts at a time (experts e0 + lane):
// entries [lo, hi) and the row tiles up to and with the lane's expert.  The
// experts are gone through from the last to the first: a group ends at the
// smallest offset behind its start's, so that groups never share an entry,
// whatever the offsets are.
struct Groups {
    int32_t lo, hi, incl;
    int64_t total;  // tiles of all experts
};

// Loads the groups of experts e0 ..; `least` is the smallest offset behind
// them (maxEntries at first) and becomes that behind e0 - 1's start.
template <int BM>
__device__ __forceinline__ void load_groups(const ProductParams &P, int32_t e0, int32_t &least, Groups &g) {
    const int lane = threadIdx.x & 63, e = e0 + lane;
    int32_t end = e < P.E ? min(max(P.offsets[e + 1], 0), P.maxEntries) : P.maxEntries;
    g.lo = e < P.E ? min(max(P.offsets[e], 0), P.maxEntries) : P.maxEntries;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_down(end, d);
        if (lane + d < 64) end = min(end, o);
    }
    end = min(end, least);
    g.hi = e < P.E ? max(end, g.lo) : g.lo;
    g.incl = wave_incl_scan((g.hi - g.lo + BM - 1) / BM);
    least = uniform(min(end, g.lo));  // of lane 0
}

template <int BM>
__device__ __forceinline__ Groups count_tiles(const ProductParams &P, int32_t NT) {
    Groups g;
    int64_t total = 0;
    int32_t least = P.maxEntries;
    for (int32_t e0 = (P.E - 1) & ~63; e0 >= 0; e0 -= 64) {
        load_groups<BM>(P, e0, least, g);
        total += uniform(__shfl(g.incl, 63));
    }
    g.total = total * NT;
    return g;
}

// Tile b among all experts' tiles (BM entries x BN columns), or e = -1 when
// there are fewer.  Each XCD (block b % 8) takes a contiguous stretch of the
// tiles, so the tiles that run on it together share operands in its L2;
// within an expert, bands of four row tiles (up to seven where four would
// leave a rest) go through the columns together.
template <int BM, int BN>
__device__ __forceinline__ TileAt find_tile(const ProductParams &P, Groups &g, int32_t NT, int32_t b) {
    const int64_t per = (g.total + 7) / 8;
    const int64_t at = (b & 7) * per + (b >> 3);
    TileAt t{-1, 0, 0, 0};
    if ((b >> 3) >= per || at >= g.total) return t;
    int64_t before = 0;
    int32_t least = P.maxEntries;
    for (int32_t e0 = (P.E - 1) & ~63; e0 >= 0; e0 -= 64) {
        if (P.E > 64) load_groups<BM>(P, e0, least, g);
        const uint64_t past = __ballot((before + g.incl) * NT > at);
        if (past) {
            const int f = __builtin_ctzll(past);
            const int32_t lo = __builtin_amdgcn_readlane(g.lo, f), hi = __builtin_amdgcn_readlane(g.hi, f);
            const int32_t tiles = (hi - lo + BM - 1) / BM;
            const int32_t r0 = (int32_t)(at - (before + __builtin_amdgcn_readlane(g.incl, f) - tiles) * NT);  // inside the expert
            const int32_t size = ceil_div(tiles, max(tiles >> 2, 1));  // row tiles of a band
            const int32_t band = r0 / (size * NT), rows = min(size, tiles - band * size), r = r0 - band * size * NT;
            const int32_t n = r / rows, m = band * size + r - n * rows;
            t = TileAt{uniform(e0 + f), uniform(lo + m * BM), uniform(min(hi, lo + m * BM + BM)), uniform(n * BN)};
            return t;
        }
        before += uniform(__shfl(g.incl, 63));
    }
    return t;
}

// Few entries per expert: the weights are streamed once, at the rate of the
// memory.  A block takes 16 FN columns and 16 FM entries of one expert; its
// four waves share the row's elements out among them (256-element chunks in
// turn) and add their sums up at the end, in LDS, in wave order.  No wave needs
// another's operands, so they go straight from memory into registers, DEPTH
// chunks ahead, with no barrier on the way.
//
// A lane's scale byte is byte l / 16 of its row's word: one shift.
template <int FM, int FN, int DEPTH, bool OUT32>
__global__ __launch_bounds__(256) void product_stream_kernel(ProductParams P) {
    constexpr int BM = 16 * FM, BN = 16 * FN;
    __shared__ __attribute__((aligned(16))) float part[4][BM][BN + 4];  // + 4: rows on other banks
    __shared__ int32_t rows[BM];
    const int32_t NT = ceil_div(P.N, BN);
    Groups groups = count_tiles<BM>(P, NT);
    const TileAt T = find_tile<BM, BN>(P, groups, NT, blockIdx.x);
    if (T.e < 0) return;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int r16 = lane & 15, kb = lane >> 4;
    const uint8_t *m[FM], *ms[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        const int32_t ent = min(T.m0 + f * 16 + r16, T.hi - 1);
        const int32_t r = P.entryRow ? P.entryRow[ent] : ent;
        const bool in = (uint32_t)r < (uint32_t)P.numRows;
        if (wave == 0 && kb == 0) rows[f * 16 + r16] = in ? r : -1;
        m[f] = P.rows + (int64_t)(in ? r : 0) * P.rowBytes + kb * 16;
        ms[f] = P.rowScales + (int64_t)(in ? r : 0) * P.words * 4;
    }
    uint32_t n[FN], ns[FN];
    const int64_t first = (int64_t)T.e * P.N + T.n0;
    const __amdgpu_buffer_rsrc_t nrs = buffer_of(P.weights + first * P.rowBytes), nsrs = buffer_of(P.weightScales + first * P.words * 4);
#pragma unroll
    for (int f = 0; f < FN; ++f) {
        const int32_t c = min(f * 16 + r16, P.N - 1 - T.n0);
        n[f] = (uint32_t)(c * P.rowBytes + kb * 16);
        ns[f] = (uint32_t)(c * P.words * 4);
    }
    struct Chunk {
        u32x4 m[FM][2], n[FN][2];
        u32x2 sm[FM], sn[FN];
    };
    auto load = [&](Chunk &c, int at) {  // chunk `at`, whole
        const int k = uniform(at * 128), w = uniform(at * 8);
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            c.n[f][0] = __builtin_amdgcn_raw_buffer_load_b128(nrs, (int)n[f], k, 0);
            c.n[f][1] = __builtin_amdgcn_raw_buffer_load_b128(nrs, (int)n[f] + 64, k, 0);
            c.sn[f] = __builtin_amdgcn_raw_buffer_load_b64(nsrs, (int)ns[f], w, 0);
        }
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            c.m[f][0] = load16<false>(m[f] + k);
            c.m[f][1] = load16<false>(m[f] + k + 64);
            c.sm[f] = *reinterpret_cast<const u32x2_dword *>(ms[f] + w);
        }
    };
    auto load_tail = [&](Chunk &c, int at) {  // the last chunk, which the rows end in: zeros behind their end
        const int k = at * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool in = k + h * 64 + kb * 16 < P.rowBytes;
            const int32_t word = min(at * 2 + h, P.words - 1) * 4;
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                c.n[f][h] = __builtin_amdgcn_raw_buffer_load_b128(nrs, in ? (int)n[f] + h * 64 + k : (int)n[f] - kb * 16, 0, 0);
                const uint32_t v = __builtin_amdgcn_raw_buffer_load_b32(nsrs, (int)ns[f] + word, 0, 0);
                c.sn[f][h] = in ? v : 0x7f7f7f7fu;
            }
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const u32x4 v = load16<false>(in ? m[f] + h * 64 + k : m[f] - kb * 16);
                c.m[f][h] = in ? v : u32x4{0, 0, 0, 0};
                const uint32_t s = *reinterpret_cast<const uint32_t *>(ms[f] + word);
                c.sm[f][h] = in ? s : 0x7f7f7f7fu;
            }
        }
    };
    f32x4 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    auto multiply = [&](const Chunk &c) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    acc[i][j] = mfma_fp4<0, 0>(c.n[i][h], c.m[j][h], acc[i][j], (int32_t)(c.sn[i][h] >> (8 * kb)),
                                               (int32_t)(c.sm[j][h] >> (8 * kb)));
    };
    const int whole = P.rowBytes / 128;                        // whole chunks
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
    if (P.rowBytes % 128 != 0 && (whole & 3) == wave) {
        load_tail(c[0], whole);
        multiply(c[0]);
    }
    // lane: entry r16 of fragment j, columns 4 kb .. + 3 of fragment i
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) *reinterpret_cast<f32x4 *>(&part[wave][j * 16 + r16][i * 16 + kb * 4]) = acc[i][j];
    __syncthreads();
    constexpr int kPer = OUT32 ? 4 : 8;  // columns per thread: 16 bytes of results
    for (int u = threadIdx.x; u < BM * BN / kPer; u += 256) {
        const int ent = u / (BN / kPer), col = (u - ent * (BN / kPer)) * kPer;
        if (T.m0 + ent >= T.hi || T.n0 + col >= P.N) continue;
        float v[kPer];
        const bool none = rows[ent] < 0;  // a row of zeros
        const float w = P.entryWeight ? P.entryWeight[T.m0 + ent] : 1.0f;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            v[q] = ((part[0][ent][col + q] + part[1][ent][col + q]) + part[2][ent][col + q]) + part[3][ent][col + q];
            v[q] = none ? 0.0f : v[q] * w;
        }
        const int64_t o = (int64_t)(T.m0 + ent) * P.N + T.n0 + col;
        if constexpr (OUT32)
            *reinterpret_cast<f32x4 *>(static_cast<float *>(P.out) + o) = f32x4{v[0], v[1], v[2], v[3]};
        else
            *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(P.out) + o) =
                u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
    }
}

// A BM x BN tile by four waves, each (BM/2) x (BN/2); the weights are the
// instruction's rows, the entries its columns, so a lane ends with runs of 8
// consecutive output columns of one entry.
//
// Steps of 256 elements (128 bytes a row) go through two LDS buffers, loaded
// by the memory pipeline itself (no registers on the way).  A step is two
// halves of 128 elements; the operands of a half are read into registers
// during the half before:
//     read half 1 of step k        | products of half 0
//     wait: step k+1 has arrived (requested one whole step ago); barrier
//     request step k+2 into step k's buffer
//     read half 0 of step k+1      | products of half 1
// LDS rows are 128 bytes: the 16-byte pieces of a row are stored at piece ^
// (row's place among eight), so that the 16 lanes that read one piece of 16
// rows spread over all banks.
// Scale bytes: a thread takes one word (128 elements of a row) of the four rows
// that sit at its place in four fragments, and turns the 4 x 4 bytes over, so
// that a lane finds the bytes of four fragments in one word of LDS; which of
// the four a product takes is part of the instruction.  4 words a row cover
// two steps, so this happens every other step.
// A block goes on to its next tile (a stride of the grid further) by itself:
// the first steps of that are requested before this one's results are stored.
//
// WIDE: the array of rows passes 32-bit offsets.
template <int BM, int BN, bool OUT32, bool WIDE>
__global__ __launch_bounds__(256, BM *BN > 128 * 128 ? 1 : 2) void product_tile_kernel(ProductParams P) {
    constexpr int FM = BM / 32, FN = BN / 32;      // 16-wide fragments of a wave
    constexpr int LM = BM / 32, LN = BN / 32;      // LDS loads of a wave per step (8 rows each)
    constexpr int kQuads = (BM + BN) / 64;         // four fragments each, the rows' first
    constexpr int SQ = kQuads / 4;                 // of which a wave stages the scales
    __shared__ __attribute__((aligned(16))) uint8_t mbuf0[BM * 128], mbuf1[BM * 128], nbuf0[BN * 128], nbuf1[BN * 128];
    // scale bytes [step pair][word][byte][quad][row in the fragment][fragment of the four]
    __shared__ __attribute__((aligned(16))) uint32_t sc[2][4][4][kQuads][16];
    // of this and the next tile: the entries' rows (-1: none of the array's) and weights
    __shared__ int32_t rows[2][BM];
    __shared__ float factor[2][BM];
    const int32_t NT = ceil_div(P.N, BN);
    Groups groups = count_tiles<BM>(P, NT);
    int32_t b = blockIdx.x;
    TileAt T = find_tile<BM, BN>(P, groups, NT, b);
    if (T.e < 0) return;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int r16 = lane & 15, kb = lane >> 4;
    const int wm = (wave & 1) * (BM / 2), wn = (wave >> 1) * (BN / 2);

    // The lane again, opaque: what is computed from it is computed there, not kept in registers from tile to tile.
    auto fresh = [&] {
        int l = lane;
        asm volatile("" : "+v"(l));
        return l;
    };
    // A tile's rows and weights, on the way to LDS.  Entries behind the tile's last repeat it.
    int32_t row = -1;
    float weight = 1.0f;
    auto look = [&](const TileAt &t) {
        const int tid = wave * 64 + fresh();
        if (tid >= BM) return;
        const int32_t ent = min(t.m0 + tid, t.hi - 1);
        row = P.entryRow ? P.entryRow[ent] : ent;
        if (P.entryWeight) weight = P.entryWeight[ent];
    };
    auto keep = [&](int par) {
        const int tid = wave * 64 + fresh();
        if (tid >= BM) return;
        rows[par][tid] = (uint32_t)row < (uint32_t)P.numRows ? row : -1;
        factor[par][tid] = weight;
    };
    // The 16-byte piece of a row that lane l requests: of the tile's rows, and of its columns in even loads (in odd
    // ones ^ 64).
    auto piece_m = [](int l) { return ((l & 7) ^ (l >> 3)) * 16; };
    auto piece_n = [](int l) { return ((l & 7) ^ ((l >> 3) & 3)) * 16; };
    // Offsets of what this lane requests in a step: of the rows (their index where offsets pass 32 bits), and of the
    // columns from the tile's first; and those of the scale words it stages.
    uint32_t mat[LM], nat[LN], sat[SQ][4];
    const int sword = lane & 3, sslot = lane >> 2;  // the word and the row in its fragment that it stages
    const uint8_t *nbase, *nsbase;
    auto set_tile = [&](const TileAt &t, int par) {
        const int ln = fresh();
        const int srow = ln >> 2;
        nbase = P.weights + ((int64_t)t.e * P.N + t.n0) * P.rowBytes;
        nsbase = P.weightScales + ((int64_t)t.e * P.N + t.n0) * P.words * 4;
#pragma unroll
        for (int i = 0; i < LM; ++i) {
            mat[i] = (uint32_t)max(rows[par][wave * (BM / 4) + i * 8 + (ln >> 3)], 0);
            if (!WIDE) mat[i] = mat[i] * (uint32_t)P.rowBytes + piece_m(ln);
        }
#pragma unroll
        for (int q = 0; q < SQ; ++q) {
            const int quad = q * 4 + wave;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                if (quad < BM / 64) {
                    sat[q][f] = (uint32_t)max(rows[par][quad * 64 + f * 16 + srow], 0);
                } else {
                    const int n = (quad - BM / 64) * 64 + (f >> 1) * 32 + (srow >> 2) * 8 + (f & 1) * 4 + (srow & 3);
                    sat[q][f] = (uint32_t)min(n, P.N - 1 - t.n0);
                }
                if (!WIDE) sat[q][f] *= (uint32_t)P.words * 4;
            }
        }
#pragma unroll
        for (int i = 0; i < LN; ++i)
            nat[i] = (uint32_t)(min(wave * (BN / 4) + i * 8 + (ln >> 3), P.N - 1 - t.n0) * P.rowBytes) + (piece_n(ln) ^ (i & 1) * 64);
    };
    const __amdgpu_buffer_rsrc_t mrs = buffer_of(P.rows);
    const int NK = (P.rowBytes + 127) / 128, blocks = P.H / 32;
    const int tail = NK * 128 - P.rowBytes;  // bytes of the last step behind the rows' end

    // Load t of the wave's LM + LN in step k.  Pieces behind the end of the rows repeat the last one (clear_tail).
    auto request = [&](auto t, int step, uint8_t *mb, uint8_t *nb) {
        const int k = uniform(step);
        constexpr int I = decltype(t)::value;
        int w = wave;  // opaque: the place is added up here, not kept in 16 scalar registers
        asm volatile("" : "+s"(w));
        if constexpr (I < LM) {
            uint8_t *to = mb + (w * (BM / 4) + I * 8) * 128;
            if constexpr (WIDE)
                load_lds16(P.rows + ((uint64_t)mat[I] * (uint32_t)P.rowBytes + (uint32_t)(k * 128 + piece_m(lane))), to);
            else
                load_lds16(mrs, mat[I], k * 128, to);
        } else {
            load_lds16(buffer_of(nbase), nat[I - LM], k * 128, nb + (w * (BN / 4) + (I - LM) * 8) * 128);
        }
    };
    auto request_last = [&](uint8_t *mb, uint8_t *nb) {  // step NK - 1, which the rows may end in
        const int at = uniform((NK - 1) * 128), last = 112 - tail;  // the last piece there is
        const int ln = fresh(), m = piece_m(ln), n0 = piece_n(ln), n1 = n0 ^ 64;
        each<LM>([&](auto t) {
            constexpr int I = decltype(t)::value;
            uint8_t *to = mb + (wave * (BM / 4) + I * 8) * 128;
            if constexpr (WIDE)
                load_lds16(P.rows + ((uint64_t)mat[I] * (uint32_t)P.rowBytes + (uint32_t)(at + min(m, last))), to);
            else
                load_lds16(mrs, mat[I] - m + min(m, last), at, to);
        });
        each<LN>([&](auto t) {
            constexpr int I = decltype(t)::value;
            const int own = I & 1 ? n1 : n0;
            load_lds16(buffer_of(nbase), nat[I] - own + min(own, last), at, nb + (wave * (BN / 4) + I * 8) * 128);
        });
    };
    // Rows that end inside the last step: zeros in the entries' pieces behind the end, once they have arrived.
    // (The weights' pieces there hold finite values and scales: nothing adds up.)
    auto clear_tail = [&](uint8_t *mb) {
        if (tail == 0) return;
        const int ln = fresh();
#pragma unroll
        for (int t = 0; t < LM; ++t)
            if (piece_m(ln) >= 128 - tail)
                *reinterpret_cast<u32x4 *>(mb + wave * (BM / 4) * 128 + t * 1024 + ln * 16) = u32x4{0, 0, 0, 0};
        __syncthreads();
    };
    struct Words {
        uint32_t w[SQ][4];
    };
    Words sreg;  // the next pair of steps' scale words, on the way to LDS
    auto scales_load = [&](Words &sreg, int pair) {  // words 4 pair .. + 3, behind the rows' end the last one again
        const uint32_t at = (uint32_t)min(pair * 4 + sword, P.words - 1) * 4;
#pragma unroll
        for (int q = 0; q < SQ; ++q) {
            const uint8_t *base = q * 4 + wave < BM / 64 ? P.rowScales : nsbase;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                if constexpr (WIDE)
                    sreg.w[q][f] = *reinterpret_cast<const uint32_t *>(base + ((uint64_t)sat[q][f] * ((uint32_t)P.words * 4) + at));
                else
                    sreg.w[q][f] = __builtin_amdgcn_raw_buffer_load_b32(buffer_of(base), (int)(sat[q][f] + at), 0, 0);
            }
        }
    };
    auto scales_arrived = [&](Words &sreg, int pair) {  // 127 behind the rows' last block
        const int left = blocks - (pair * 4 + sword) * 4;  // blocks of this word
        const uint32_t keep = left >= 4 ? 0xffffffffu : left > 0 ? (1u << (left * 8)) - 1 : 0u;
#pragma unroll
        for (int q = 0; q < SQ; ++q)
#pragma unroll
            for (int f = 0; f < 4; ++f) sreg.w[q][f] = (sreg.w[q][f] & keep) | (0x7f7f7f7fu & ~keep);
    };
    auto scale_store = [&](auto j, const Words &sreg, int pair) {  // byte b of the four rows' words: one of the 4 SQ words this thread stages
        constexpr int q = decltype(j)::value / 4, b = decltype(j)::value % 4;
        const uint32_t lo = __builtin_amdgcn_perm(sreg.w[q][1], sreg.w[q][0], (uint32_t)(b | (b + 4) << 8 | 0x0c0c0000));
        const uint32_t hi = __builtin_amdgcn_perm(sreg.w[q][3], sreg.w[q][2], (uint32_t)(b << 16 | (b + 4) << 24 | 0x0c0c));
        sc[pair & 1][sword][b][q * 4 + wave][sslot] = lo | hi;
    };

    struct Half {
        u32x4 m[FM], n[FN];
    };
    struct Scales {  // of both halves of a step
        int32_t m[2][FM / 4], n[2][FN / 4];
    };
    // lane's row inside a fragment: entries in order; columns so that fragments 2p and 2p + 1 of a lane join to
    // eight in a row: column 32 p + 8 (r / 4) + 4 (f & 1) + r % 4
    const int mrow = wm + r16, nrow = wn + (r16 >> 2) * 8 + (r16 & 3);
    const int msw = r16 & 7, nsw = (r16 & 3) | (((r16 >> 2) & 1) << 2);
    auto read_scales = [&](Scales &s, int k) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint32_t(*sp)[16] = sc[(k >> 1) & 1][(k & 1) * 2 + half][kb];
#pragma unroll
            for (int q = 0; q < FN / 4; ++q) s.n[half][q] = (int32_t)sp[(BM + wn) / 64 + q][r16];
#pragma unroll
            for (int q = 0; q < FM / 4; ++q) s.m[half][q] = (int32_t)sp[wm / 64 + q][r16];
        }
    };
    constexpr int kReads = FM + FN;
    // LDS read r of half `half` of a step, in the order in which the products need them.
    auto read = [&](auto r, Half &h, const uint8_t *mb, const uint8_t *nb, int half) {
        constexpr int R = decltype(r)::value;
        if constexpr (R >= 1 && R <= FN) {
            constexpr int F = R - 1;
            h.n[F] = *reinterpret_cast<const u32x4 *>(nb + nrow * 128 + (((half * 4 + kb) ^ nsw) * 16) +
                                                      ((F >> 1) * 32 + (F & 1) * 4) * 128);
        } else {
            constexpr int F = R == 0 ? 0 : R - FN;
            h.m[F] = *reinterpret_cast<const u32x4 *>(mb + mrow * 128 + (((half * 4 + kb) ^ msw) * 16) + F * 16 * 128);
        }
    };
    f32x4 acc[FN][FM];
    // The products of half HALF of a step, one matrix instruction after the other; dealt out between them, where the
    // matrix instructions leave issue slots: the reads of the next half from mb and nb, and, by WITH, the requests of
    // step rk into rmb and rnb, where rk begins a pair of steps after its scales have gone into LDS and the next pair's
    // have been asked for.
    auto multiply = [&](auto half, auto with, const Half &h, const Scales &s, Half &next, const uint8_t *mb, const uint8_t *nb,
                        int rk, uint8_t *rmb, uint8_t *rnb) {
        constexpr int HALF = decltype(half)::value, WITH = decltype(with)::value, kAll = FM * FN;
        each<kAll>([&](auto q) {
            constexpr int Q = decltype(q)::value, J = Q / FN, I = Q % FN;
            mfma_fp4_inplace<I & 3, J & 3>(acc[I][J], h.n[I], h.m[J], s.n[HALF][I >> 2], s.m[HALF][J >> 2]);
            constexpr int kGap = kAll / (kReads + 1) ? kAll / (kReads + 1) : 1;
            if constexpr (Q % kGap == 0 && Q / kGap < kReads) read(Const<Q / kGap>{}, next, mb, nb, 1 - HALF);
            // requests after the stores of the scales: those would wait for requests under way (to other parts of LDS,
            // which the compiler does not tell apart)
            constexpr int kFrom = WITH == kTurn ? kAll / 4 : 0, kReqGap = (kAll - kFrom) / (LM + LN);
            if constexpr (WITH == kTurn && Q == 0) scales_arrived(sreg, rk >> 1);
            if constexpr (WITH == kTurn && Q < kFrom && Q % (kFrom / (4 * SQ)) == 0)
                scale_store(Const<Q / (kFrom / (4 * SQ))>{}, sreg, rk >> 1);
            if constexpr (WITH == kTurn && Q == kFrom - 1) scales_load(sreg, (rk >> 1) + 1);
            if constexpr (WITH != 0 && Q >= kFrom && (Q - kFrom) % kReqGap == kReqGap / 2 && (Q - kFrom) / kReqGap < LM + LN)
                request(Const<(Q - kFrom) / kReqGap>{}, rk, rmb, rnb);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    using First = Const<0>;
    using Second = Const<1>;
    using Alone = Const<0>;
    using Request = Const<kRequest>;
    using Turn = Const<kTurn>;
    // This wave's LDS reads are in its registers and all but its last `left` requests (loads, and stores of results)
    // are done; then all waves' are.
    auto meet = [&](auto left) {
        constexpr int L = decltype(left)::value;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((L & 15) | (L >> 4) << 14 | 0x70);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    using All = Const<0>;

    Half h0, h1;
    Scales s0, s1;  // of even and odd steps
    Words sfirst;
    auto request_first = [&] {  // the tile's first two steps and the scales of its first four
        scales_load(sfirst, 0);
        if (NK == 1) {
            request_last(mbuf0, nbuf0);
        } else {
            each<LM + LN>([&](auto t) { request(t, 0, mbuf0, nbuf0); });
            if (NK == 2)
                request_last(mbuf1, nbuf1);
            else
                each<LM + LN>([&](auto t) { request(t, 1, mbuf1, nbuf1); });
        }
        scales_load(sreg, 1);
    };
    // Stores of results per wave and tile, whatever the tile holds: they stay under way while the next tile begins.
    constexpr int kStores = FM * FN / 2 * (OUT32 ? 2 : 1), kStoresLeft = kStores < 63 ? kStores : 63;
    // A tile's sums begin at zero, its first scales go into LDS.
    auto begin = [&] {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                acc[i][j] = f32x4{0, 0, 0, 0};
                asm volatile("" : "+a"(acc[i][j]));
            }
        scales_arrived(sfirst, 0);
        each<4 * SQ>([&](auto j) { scale_store(j, sfirst, 0); });
    };
    // For the compiler: the words on the way have arrived here (it would wait for later stores too).
    auto settle = [&] {
#pragma unroll
        for (int q = 0; q < SQ; ++q)
#pragma unroll
            for (int f = 0; f < 4; ++f) asm volatile("" : "+v"(sreg.w[q][f]));
    };
    look(T);
    keep(0);
    meet(All{});
    set_tile(T, 0);
    request_first();
    begin();
    meet(All{});
    settle();
    for (int par = 0;; par ^= 1) {
    if (NK == 1) clear_tail(mbuf0);
    b += gridDim.x;
    const TileAt next = find_tile<BM, BN>(P, groups, NT, b);
    if (next.e >= 0) look(next);
    read_scales(s0, 0);
    each<kReads>([&](auto r) { read(r, h0, mbuf0, nbuf0, 0); });
    int k = 0;
    for (; k + 4 < NK; k += 2) {  // steps k and k + 1; k + 2 and k + 3, requested here, are not the last
        multiply(First{}, Alone{}, h0, s0, h1, mbuf0, nbuf0, 0, mbuf0, nbuf0);
        if (k == 0)
            meet(Const<63>{});  // step 1 was there already: no wait for the results' stores
        else
            meet(All{});
        read_scales(s1, k + 1);
        multiply(Second{}, Turn{}, h1, s0, h0, mbuf1, nbuf1, k + 2, mbuf0, nbuf0);
        multiply(First{}, Alone{}, h0, s1, h1, mbuf1, nbuf1, 0, mbuf0, nbuf0);
        meet(All{});
        settle();
        read_scales(s0, k + 2);
        multiply(Second{}, Request{}, h1, s1, h0, mbuf0, nbuf0, k + 3, mbuf1, nbuf1);
    }
    if (next.e >= 0) keep(par ^ 1);
    // The last one to four steps, k first.  What is read behind the last step is not used.
    for (;; k += 2) {
        multiply(First{}, Alone{}, h0, s0, h1, mbuf0, nbuf0, 0, mbuf0, nbuf0);
        meet(All{});
        if (k + 2 == NK) clear_tail(mbuf1);
        read_scales(s1, k + 1);
        if (k + 2 < NK) {
            scales_arrived(sreg, (k >> 1) + 1);
            each<4 * SQ>([&](auto j) { scale_store(j, sreg, (k >> 1) + 1); });
            scales_load(sreg, (k >> 1) + 2);
            if (k + 3 == NK)
                request_last(mbuf0, nbuf0);
            else
                each<LM + LN>([&](auto t) { request(t, k + 2, mbuf0, nbuf0); });
        }
        multiply(Second{}, Alone{}, h1, s0, h0, mbuf1, nbuf1, 0, mbuf0, nbuf0);
        if (k + 1 >= NK) break;
        multiply(First{}, Alone{}, h0, s1, h1, mbuf1, nbuf1, 0, mbuf0, nbuf0);
        meet(All{});
        if (k + 3 == NK) clear_tail(mbuf0);
        read_scales(s0, k + 2);
        if (k + 4 == NK) request_last(mbuf1, nbuf1);
        multiply(Second{}, Alone{}, h1, s1, h0, mbuf0, nbuf0, 0, mbuf0, nbuf0);
        if (k + 2 >= NK) break;
    }
    mfma_done();

    // No wave needs this tile's LDS any more (all passed the last meeting): the next tile's first steps.
    if (next.e >= 0) {
        set_tile(next, par ^ 1);
        request_first();
    }
    __builtin_amdgcn_sched_barrier(0);
    // Results: stores through a buffer that ends with the tile's last entry; columns past N are sent beyond it.
    const int ln = fresh(), mfirst = wm + (ln & 15), nfirst = T.n0 + wn + (ln >> 4) * 8;
    const int32_t rowOut = P.N * (OUT32 ? 4 : 2);
    const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(
        static_cast<uint8_t *>(P.out) + (int64_t)T.m0 * rowOut, 0, (T.hi - T.m0) * rowOut, 0x00020000);
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const float w = factor[par][mfirst + j * 16];
        const bool none = rows[par][mfirst + j * 16] < 0;
#pragma unroll
        for (int p = 0; p < FN / 2; ++p) {
            float v[8];
            asm volatile("" : "+a"(acc[2 * p][j]), "+a"(acc[2 * p + 1][j]));  // not copied out before they are needed
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = acc[2 * p + (i >> 2)][j][i & 3] * w;
            if (__any(none)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = none ? 0.0f : v[i];
            }
            const int32_t n = nfirst + p * 32;
            const int32_t at = (mfirst + j * 16) * rowOut + n * (OUT32 ? 4 : 2), outside = 0x7ffffff0;
            if (OUT32) {
                __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                                             __float_as_uint(v[3])}, out, n < P.N ? at : outside, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                                                             __float_as_uint(v[7])}, out, n + 4 < P.N ? at + 16 : outside, 0, 0);
            } else {
                __builtin_amdgcn_raw_buffer_store_b128(
                    u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])}, out,
                    n < P.N ? at : outside, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (next.e < 0) return;
    T = next;
    begin();
    meet(Const<kStoresLeft>{});
    settle();
    }
}

template <int BM, int BN, bool WIDE>
hipError_t launch_tiles(const ProductParams &P, bool out32, hipStream_t stream) {
    // row tiles at most: one partly filled for each expert
    const int64_t tiles = ((int64_t)P.maxEntries / BM + (P.E < P.maxEntries ? P.E : P.maxEntries)) * ceil_div(P.N, BN);
    if (tiles > INT32_MAX / 2) return hipErrorInvalidConfiguration;
    int device = 0, cus = 0;
    hipError_t err = hipGetDevice(&device);
    if (err == hipSuccess) err = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device);
    if (err != hipSuccess) return err;
    // as many blocks as run at once, a multiple of the 8 XCDs
    const int64_t most = (int64_t)ceil_div(cus * (BM * BN > 128 * 128 ? 1 : 2), 8) * 8, blocks = (tiles + 7) / 8 * 8;
    const dim3 grid((uint32_t)(blocks < most ? blocks : most));
    if (out32)
        hipLaunchKernelGGL((product_tile_kernel<BM, BN, true, WIDE>), grid, dim3(256), 0, stream, P);
    else
        hipLaunchKernelGGL((product_tile_kernel<BM, BN, false, WIDE>), grid, dim3(256), 0, stream, P);
    return hipGetLastError();
}

template <int FM, int FN, int DEPTH>
hipError_t launch_stream(const ProductParams &P, bool out32, hipStream_t stream) {
    const int64_t tiles = ((int64_t)P.maxEntries / (16 * FM) + (P.E < P.maxEntries ? P.E : P.maxEntries)) * ceil_div(P.N, 16 * FN);
    const int64_t blocks = (tiles + 7) / 8 * 8;
    if (blocks > (1 << 23)) return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)blocks);
    if (out32)
        hipLaunchKernelGGL((product_stream_kernel<FM, FN, DEPTH, true>), grid, dim3(256), 0, stream, P);
    else
        hipLaunchKernelGGL((product_stream_kernel<FM, FN, DEPTH, false>), grid, dim3(256), 0, stream, P);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_product(const ProductParams &P, bool out32, hipStream_t stream) {
    if (P.maxEntries == 0) return hipSuccess;
    switch (plan_product(P.E, P.N, P.H, P.maxEntries, P.numRows)) {
    case kProductStream16: return launch_stream<1, 2, 3>(P, out32, stream);
    case kProductStream64: return launch_stream<4, 2, 2>(P, out32, stream);
    case kProductTiles128: return launch_tiles<128, 128, false>(P, out32, stream);
    case kProductTiles128Wide: return launch_tiles<128, 128, true>(P, out32, stream);
    case kProductTiles256: return launch_tiles<256, 256, false>(P, out32, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace epdc
