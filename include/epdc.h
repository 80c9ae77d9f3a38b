/*
 * epdc.h -- C ABI of libepdc.so: one source rank's share of MoE
 * expert-parallel token dispatch and combine on one MI355X (gfx950).
 *
 * Operations (definitions from the pages):
 *   dispatch  COUNT -> SCAN -> FINALIZE.  mori PR #599 "Perf/ep disp 1250
 *             ship", items "ballot dedup" and "cached destPe/keep + deferred
 *             null write": each (token, top-k slot) maps to a destination PE;
 *             a token reaches each PE at most once; the rows and per-token
 *             metadata are written into per-PE receive windows and every
 *             dropped slot gets a 4-byte null entry.  Dispatch only moves bytes
 *             (MORI JIT v2 design doc, §3.7).
 *   combine   MORI JIT v2 design doc, §5 and §9: a gather combine -- each token
 *             pulls the rows its PEs returned and reduces them.
 *   scatter combine (push + reduce)  MORI JIT v2 design doc, §5 and §9 (the
 *             FlyDSL backend's scatter combine) with the landing rows sized
 *             in the aiter MegaMoE commits on the mori PR #599 page: each
 *             destination pushes its returned rows into per-(token, PE)
 *             landing rows at offsets the dispatch hands over, then the
 *             source reduces them.  Same result as the gather combine.
 *
 *   routing, fp4x2 quantisation, grouping by expert, the experts' product
 *             What stands on both sides of a dispatch and a combine: the
 *             top-k experts and weights of a token (and their gradient), the
 *             fp4x2 wire's codes and scales, the expert-sorted list of a
 *             window's rows, and the product of those rows with each expert's
 *             fp4x2 weights.  Declared in the second half of this file.
 *
 * Argument names follow EpCfg (MORI JIT v2 design doc, §3.2).  The geometry
 * fields of EpCfg (blockNum, warpPerBlock, waveSize) are not part of the ABI:
 * the library picks launch geometry itself.
 *
 * Conventions for every entry point:
 *   - Every pointer named "device" is device memory owned by the caller; the
 *     library allocates nothing, copies nothing to the host and never
 *     synchronises.  Calls are asynchronous on `stream`, so they can be
 *     captured into a HIP graph.  `stream` is a hipStream_t passed as void *
 *     (NULL is the default stream): the header then compiles without the HIP
 *     headers, and a hipStream_t converts to it implicitly.
 *   - All checks run on the host before any launch.  On failure a negative
 *     EPDC_ERR_* code is returned, nothing is launched, and epdc_last_error()
 *     describes the failure.  No entry point throws (MORI JIT v2 design doc,
 *     §6: every C entry point is noexcept and reports through a last-error
 *     string).
 *   - Index layout: T = numTokens, K = numExpertPerToken, W = worldSize,
 *     M = maxTokPerRank, H = hiddenDim, Epr = numExpertPerRank, E = W*Epr.
 *     All arrays are dense row-major with exactly these extents.
 *   - An array that a call writes overlaps none that it reads, and no other
 *     that it writes.
 */
#ifndef EPDC_H
#define EPDC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Row element types, numbered as the pages' EpDType (MORI JIT v2 design doc,
 * §3.7 and §7: the enum values must match the binding's table).  Dispatch
 * only moves rows, so it takes all four: bf16 (2 bytes per element), fp32 (4)
 * and the one-byte fp8 and fp4x2 (for fp4x2 one element is a byte holding
 * two e2m1 values, so hiddenDim counts bytes).  Combine sums rows, so it
 * takes only EPDC_BF16 and EPDC_FP32, for its returned rows and, chosen
 * apart, for its output (§5: the combine outputs bf16 or fp32).  A
 * narrow-wire pair (fp8 or fp4x2 dispatch, bf16 combine) is two calls with
 * two cfgs.  The quantisation scales of a narrow-wire row travel beside it as
 * per-token metadata (scaleDim, below). */
typedef enum {
    EPDC_BF16 = 0,
    EPDC_FP32 = 1,
    EPDC_FP8 = 2,
    EPDC_FP4X2 = 3
} epdc_dtype;

enum {
    EPDC_OK = 0,
    EPDC_ERR_INVALID_ARG = -1, /* a cfg field out of range, numTokens < 0, K > E, W*M too large */
    EPDC_ERR_UNSUPPORTED = -2, /* dtype not allowed on this call (see above), useWeights not 0/1 */
    EPDC_ERR_CAPACITY = -3,    /* numTokens > maxTokPerRank                                    */
    EPDC_ERR_ALIGN = -4,       /* row bytes not a multiple of 16, or a misaligned pointer      */
    EPDC_ERR_NULLPTR = -5,     /* a required pointer (or cfg) is NULL                          */
    EPDC_ERR_SCRATCH = -6,     /* scratchBytes below epdc_dispatch_scratch_bytes(cfg)          */
    EPDC_ERR_HIP = -7          /* the HIP runtime reported an error (no device, launch failed) */
};

/* Shape and options of one dispatch/combine pair (EpCfg field names).
 *   worldSize          W, 1..64 (one bit per PE in a 64-lane wavefront)
 *   hiddenDim          H elements per token row; the row, H times the element
 *                      size of dtype, must be a multiple of 16 bytes
 *   maxTokPerRank      M >= 1: capacity of x and of each receive window, in rows;
 *                      W*M must not exceed 2^31-1 (flat indices are int32)
 *   numExpertPerRank   Epr >= 1; expert e lives on PE e / Epr
 *   numExpertPerToken  K, 1..64, K <= E
 *   dtype              row element type (epdc_dtype; see above for each call)
 *   useWeights         1: dispatch copies the weights, combine applies them; 0: ignored
 *   scaleDim           S, 0..EPDC_MAX_SCALE_DIM: fp32 scales per token that the
 *                      dispatch forwards with each of the token's rows (0: none).
 *                      MORI JIT v2 design doc, §4 (the dispatch takes a `scales`
 *                      argument) and §5 (an `out_scales` region exists only when
 *                      scale_dim > 0); the mori PR #599 page's merge notes carry
 *                      the per-token scale row as a fourth metadata field beside
 *                      token index, expert ids and weights.  Combine, push and
 *                      reduce ignore it. */
typedef struct epdc_cfg {
    int32_t worldSize;
    int32_t hiddenDim;
    int32_t maxTokPerRank;
    int32_t numExpertPerRank;
    int32_t numExpertPerToken;
    int32_t dtype;
    int32_t useWeights;
    int32_t scaleDim;
} epdc_cfg;

/* Largest scaleDim: one fp32 scale per 16 elements of a 16384-wide row. */
#define EPDC_MAX_SCALE_DIM 1024

/* Bytes of device scratch epdc_dispatch needs for this cfg: a 4224-byte header
 * (completion counters and a status word) plus two 32-bit words per (64-token
 * tile, PE) of maxTokPerRank tokens -- a few KB.  Returns 0 if cfg is invalid.
 *
 * The pages' dispatch reserves rows with a cross-device fetch_add; this one
 * instead computes every row in ascending token order (so windows are stable
 * and the result deterministic) from per-tile counts that the kernel's blocks
 * exchange through this buffer: one block per 64-token tile publishes the
 * tile's count per PE and the blocks of later tiles sum them.
 *
 * The scratch must be zero-filled once before its first use (e.g. one
 * hipMemset at allocation).  Every dispatch leaves it zeroed again, so it
 * needs no reset between calls or graph replays -- except the status word.
 * One scratch buffer serves one dispatch at a time: calls that may run
 * concurrently need separate buffers. */
size_t epdc_dispatch_scratch_bytes(const epdc_cfg *cfg);

/* Status word of a dispatch scratch buffer: the 32-bit word at byte offset
 * 4 * EPDC_STATUS_WORD.  A dispatch sets it nonzero -- and never clears it --
 * when that call's outputs are invalid:
 *   EPDC_STATUS_WAIT_TIMEOUT   one of its bounded in-kernel waits gave up
 *                              (instead of hanging the GPU);
 *   EPDC_STATUS_ROW_OUTSIDE    a computed row fell outside its window (only
 *                              possible when the scratch was not zero at
 *                              launch; such rows are skipped and nothing is
 *                              written outside the windows).
 * It stays zero in correct operation.  Read it after the caller's own
 * synchronisation with the stream (one 4-byte device-to-host copy); a caller
 * that sees it nonzero discards the outputs and zeroes the scratch again. */
#define EPDC_STATUS_WORD 2
#define EPDC_STATUS_WAIT_TIMEOUT 1
#define EPDC_STATUS_ROW_OUTSIDE 2

/*
 * Dispatch numTokens tokens (0 <= numTokens <= maxTokPerRank).
 *
 * Inputs (device, read only):
 *   x            [T][H] token rows of cfg->dtype, 16-byte aligned
 *   expertIds    [T][K] int32 top-k expert ids; an id outside [0, E) marks a
 *                dropped slot (ids are not range-checked on the host)
 *   weights      [T][K] fp32; may be NULL iff useWeights == 0
 *   scales       [T][S] fp32 per-token scales (S = scaleDim); may be NULL iff S == 0
 * Outputs (device, written):
 *   recvX          [W][M][H] of cfg->dtype, 16-byte aligned: recvX[p][r] is a bitwise copy
 *                  of the r-th token (ascending token order) that reaches PE p
 *   recvTokIdx     [W][M] int32: that token's index
 *   recvExpertIds  [W][M][K] int32: that token's K expert ids
 *   recvWeights    [W][M][K] fp32: that token's K weights; NULL iff useWeights == 0
 *   recvScales     [W][M][S] fp32: that token's S scales, bitwise; NULL iff S == 0
 *   recvCount      [W] int32: rows written per PE -- stored, not accumulated
 *                  (mori PR #599 follow-up commits: the dispatch stores the
 *                  received count, so callers need no reset kernel)
 *   sendMap        [T][K] int32: for the lowest slot k of token t on PE p,
 *                  p*M + r; for every other slot (duplicate PE or invalid
 *                  id) -1, the null entry
 *   Rows r >= recvCount[p] of every window are left untouched.
 * Scratch (device): at least epdc_dispatch_scratch_bytes(cfg) bytes, 16-byte
 *   aligned, zero-filled before its first use (see above).
 * With numTokens == 0 only recvCount is written (zeros); the token-sized
 * pointers may then be NULL.
 */
int epdc_dispatch(const epdc_cfg *cfg, int32_t numTokens,
                  const void *x, const int32_t *expertIds, const float *weights, const float *scales,
                  void *recvX, int32_t *recvTokIdx, int32_t *recvExpertIds,
                  float *recvWeights, float *recvScales, int32_t *recvCount, int32_t *sendMap,
                  void *scratch, size_t scratchBytes, void *stream);

/*
 * epdc_dispatch without a caller scratch buffer, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation.  Same arguments (minus scratch and
 * scratchBytes), same kernels and bit-identical outputs.  The scratch is the
 * library's own: a 1 MiB device array per GPU, held until the process ends,
 * zeroed by a small kernel on `stream` at the first call on that device and
 * left zeroed by every call.  It allocates nothing (no hipMalloc, no library
 * allocator) on any call.
 *
 * Limit: the scratch must hold 4224 + 8 * ceil(numTokens / 64) * W' bytes (W'
 * = worldSize rounded up to a power of two), i.e. up to 130,496 tokens at 64
 * PEs, 1,044,352 at 8; beyond that the call fails with EPDC_ERR_SCRATCH and
 * launches nothing.  Calls on one GPU share its array: calls that may run at
 * the same time on that GPU (on different streams, or from several threads)
 * race and give invalid outputs -- serialise them, or use epdc_dispatch with
 * a buffer per stream.  The array's status word is not exposed.
 */
int epdc_dispatch_noalloc(const epdc_cfg *cfg, int32_t numTokens,
                          const void *x, const int32_t *expertIds, const float *weights, const float *scales,
                          void *recvX, int32_t *recvTokIdx, int32_t *recvExpertIds,
                          float *recvWeights, float *recvScales, int32_t *recvCount, int32_t *sendMap,
                          void *stream);

/*
 * Combine numTokens tokens from the rows their PEs returned.
 *
 * cfg->dtype is EPDC_BF16 or EPDC_FP32: the type of y.  outDtype is
 * EPDC_BF16 or EPDC_FP32: the type of out (either with either).
 * Inputs (device, read only):
 *   y          [W][M][H] of cfg->dtype, 16-byte aligned: returned rows, indexed like recvX
 *   expertIds  [T][K] int32, the ids given to the matching dispatch; read only
 *              when useWeights == 1 (else may be NULL)
 *   weights    [T][K] fp32 or NULL iff useWeights == 0
 *   sendMap    [T][K] int32 as written by the matching dispatch
 * Output (device): out [T][H] of outDtype, 16-byte aligned.
 *
 * For token t, the PEs of its kept slots (sendMap >= 0) are visited in
 * ascending slot order.  PE p's scale is the fp32 sum, in slot order from +0,
 * of the weights of t's slots whose valid expert lives on p (1 when
 * useWeights == 0).  acc = fmaf(scale_p, y[p][r_p][h], acc) over those PEs
 * from acc = +0 in fp32; out[t][h] = bf16_rne(acc) for a bf16 output
 * (nearest, ties to even) and acc itself for an fp32 output.  A token with no
 * kept slot yields +0.  A sendMap entry outside [0, W*M) counts as a dropped
 * slot.  Results are deterministic and bit-identical run to run.
 */
int epdc_combine(const epdc_cfg *cfg, int32_t numTokens,
                 const void *y, const int32_t *expertIds, const float *weights,
                 const int32_t *sendMap, void *out, int32_t outDtype, void *stream);

/* Landing rows of the scatter combine for numTokens tokens: numTokens *
 * min(W, K), one per (token, PE) a token can reach.  -1 if cfg (with a
 * combine dtype) or numTokens is invalid. */
int32_t epdc_landing_rows(const epdc_cfg *cfg, int32_t numTokens);

/*
 * Scatter combine, push half: what the destination PEs do.  Every window's
 * returned rows move into packed landing rows, each with a forwarded scale.
 *
 * cfg->dtype is EPDC_BF16 or EPDC_FP32: the type of y and landing.
 * numTokens is the source's token count of the matching dispatch; it sizes
 * the landing buffer (R = epdc_landing_rows(cfg, numTokens) rows).
 * Inputs (device, read only):
 *   y              [W][M][H] returned rows, indexed like recvX, 16-byte aligned
 *   recvExpertIds  [W][M][K] int32 and
 *   recvWeights    [W][M][K] fp32, as the matching dispatch wrote them; both
 *                  are read only when useWeights == 1 (else may be NULL)
 *   recvCount      [W] int32 as the matching dispatch wrote it
 * Outputs (device):
 *   landing    [R][H] of cfg->dtype, 16-byte aligned: row r < recvCount[p] of
 *              window p lands at row landOff[p] + r, landOff[p] being the sum
 *              of recvCount[q] over q < p (each count taken in [0, M]);
 *              rows from the total count on, and rows that would fall at or
 *              past R, are not written
 *   landScale  [R] fp32, written only when useWeights == 1 (else may be
 *              NULL): for each landed row, the fp32 sum, in slot order from
 *              +0, of its token's weights (recvWeights) whose valid expert
 *              (recvExpertIds) lives on p -- the scale the gather combine
 *              gives PE p for that token
 * A recvCount from the matching dispatch never exceeds R rows in total.
 */
int epdc_combine_push(const epdc_cfg *cfg, int32_t numTokens,
                      const void *y, const int32_t *recvExpertIds, const float *recvWeights,
                      const int32_t *recvCount, void *landing, float *landScale, void *stream);

/*
 * Scatter combine, reduce half: what the source does with its landing rows.
 *
 * cfg->dtype is EPDC_BF16 or EPDC_FP32: the type of landing; outDtype
 * (EPDC_BF16 or EPDC_FP32) the type of out.
 * Inputs (device, read only):
 *   landing    [R][H], landScale [R] (NULL iff useWeights == 0): as written by
 *              epdc_combine_push with the same cfg, numTokens and recvCount
 *   recvCount  [W] int32 and sendMap [T][K] int32 from the matching dispatch
 * Output (device): out [T][H] of outDtype, 16-byte aligned.
 *
 * For token t, the kept slots (sendMap >= 0) in ascending order give (p, r)
 * = (sendMap / M, sendMap % M) and so landing row landOff[p] + r;
 * acc = fmaf(scale, landing[row][h], acc) from +0 in fp32, scale = landScale
 * of that row (1 when useWeights == 0); out as in epdc_combine.  This is the
 * gather combine's order and arithmetic, so out is bit-identical to
 * epdc_combine's on the same rows.  A slot whose row lies outside the landed
 * rows (or outside [0, W*M)) counts as dropped.
 */
int epdc_combine_reduce(const epdc_cfg *cfg, int32_t numTokens,
                        const void *landing, const float *landScale, const int32_t *recvCount,
                        const int32_t *sendMap, void *out, int32_t outDtype, void *stream);

/* ------------------------------------------------------------------------
 * Routing
 * ------------------------------------------------------------------------ */

/* How logits become scores. */
typedef enum {
    EPDC_SOFTMAX = 0, /* s = exp(l - max l) / sum over the token's experts */
    EPDC_SIGMOID = 1  /* s = 1 / (1 + exp(-l))                             */
} epdc_score;

/* Largest numExperts of a router. */
#define EPDC_MAX_ROUTE_EXPERTS 1024

/* A router.
 *   numExperts         E, 1..EPDC_MAX_ROUTE_EXPERTS
 *   numExpertPerToken  K, 1..64, at most groupsPerToken * E / numGroups
 *   dtype              logits' (and their gradient's) type: EPDC_BF16 or EPDC_FP32
 *   score              epdc_score
 *   numGroups          G, 1..64, divides E: group g holds experts [g*E/G, (g+1)*E/G)
 *   groupsPerToken     1..G: a token's experts come from its best groups (G: no limit)
 *   groupTop           1 or 2, at most E/G: a group's score is the sum of that many of
 *                      its best choice values
 *   renormalize        1: a token's K weights are divided by their sum; 0: not
 *   routedScale        finite; the weights are multiplied by it */
typedef struct epdc_route_cfg {
    int32_t numExperts;
    int32_t numExpertPerToken;
    int32_t dtype;
    int32_t score;
    int32_t numGroups;
    int32_t groupsPerToken;
    int32_t groupTop;
    int32_t renormalize;
    float routedScale;
} epdc_route_cfg;

/*
 * Route numTokens tokens (numTokens >= 0): their K best experts and weights.
 *
 * Inputs (device, read only):
 *   logits     [T][E] of cfg->dtype
 *   bias       [E] fp32 or NULL (zeros): added to the scores where experts are
 *              chosen, not in the weights (a bias that balances the experts)
 * Outputs (device):
 *   expertIds  [T][K] int32, best first: what epdc_dispatch takes
 *   weights    [T][K] fp32
 *
 * An expert whose logit is NaN or -inf, or whose choice value s + bias is NaN
 * or -inf, is masked: it is never chosen (a masked logit also leaves the
 * softmax's sum).  A logit of +inf takes the softmax's whole mass, shared with
 * the token's other +inf logits.  Experts are ordered by choice value s + bias
 * -- with bias NULL by the logit, of which s is an increasing function -- and
 * groups by their score (with bias NULL and groupTop 1, by their best logit;
 * members that are masked add nothing, a group of masked members is never
 * kept).  Ties go to the lower index.  The values are compared as computed in
 * 64 bits, so the choice does not depend on how a 32-bit exponential rounds.
 * Where fewer than K experts can be chosen, the slots left hold expert id -1
 * (a dropped slot for epdc_dispatch) and weight 0.
 * weights = routedScale * s, or routedScale * s / (sum of the K chosen s)
 * with renormalize (0 if that sum is 0).
 */
int epdc_route(const epdc_route_cfg *cfg, int32_t numTokens, const void *logits, const float *bias,
               int32_t *expertIds, float *weights, void *stream);

/*
 * Gradient of epdc_route's weights with respect to its logits.
 *
 * cfg's groups are ignored (the choice of experts has no gradient), and so
 * has the bias none.  Inputs (device, read only): logits [T][E] of
 * cfg->dtype; expertIds [T][K] as epdc_route gave them (an id outside [0, E),
 * or of a masked logit, is a slot with weight 0 and no gradient; an id may
 * appear in several slots); dWeights [T][K] fp32.  Output (device): dLogits
 * [T][E] of cfg->dtype, every element written.
 * With c = routedScale, g = dWeights, s the scores and r_k = s_k / (sum of the
 * token's chosen s): dLogits_i is
 *   softmax                 s_i (c g_i - sum_j c g_j s_j)  (g_i = 0 for an i not chosen)
 *   softmax, renormalize    c r_i (g_i - sum_j g_j r_j)
 *   sigmoid                 c s_i (1 - s_i) g_i
 *   sigmoid, renormalize    c r_i (1 - s_i) (g_i - sum_j g_j r_j)
 * summed over i's slots, and 0 (but for softmax without renormalize) where i
 * has none.  Computed in fp32 and rounded once (nearest, ties to even).
 * With renormalize the shares r_k are taken among the token's slots alone: for
 * softmax r_k = exp(l_k) / (sum of exp(l_j) over the slots), which is the
 * weight / c of epdc_route unless the chosen s all vanish in 64 bits, where
 * epdc_route gives weights of 0: an expert that is not in the token's slots
 * (its bias masks it, its group was not kept, its slot was dropped) has a
 * logit of +inf, or one 745 or more above all of theirs.  The gradient of such
 * a token is that of the shares all the same; it does not read the logits of
 * other experts.  To have none, give its slots id -1 or dWeights 0.
 */
int epdc_route_grad(const epdc_route_cfg *cfg, int32_t numTokens, const void *logits,
                    const int32_t *expertIds, const float *dWeights, void *dLogits, void *stream);

/* ------------------------------------------------------------------------
 * fp4x2 rows with block scales (OCP microscaling, MXFP4)
 *
 * A row of C elements (C a multiple of 32) is C/2 bytes, each two e2m1 codes
 * (sign, 2 exponent bits, 1 mantissa bit: 0 0.5 1 1.5 2 3 4 6), the first
 * element in the low half, and one scale byte b per 32 elements, worth
 * 2^(b-127) (255: NaN).  The scale bytes of a row fill S =
 * epdc_mx_scale_dim(C) 32-bit words, block i in byte i (in memory order), the
 * bytes behind the last block 127.  So a quantised row is an EPDC_FP4X2 row of
 * hiddenDim C/2 with scaleDim S: epdc_dispatch carries both as they are.
 * ------------------------------------------------------------------------ */

/* Scale words of a row of cols elements, ceil(cols / 128); -1 if cols is not a
 * positive multiple of 32, or beyond 128 * EPDC_MAX_SCALE_DIM. */
int32_t epdc_mx_scale_dim(int32_t cols);

/*
 * Quantise rows.  x is [numWindows][rowsPerWindow][cols] of dtype (EPDC_BF16
 * or EPDC_FP32, 16-byte aligned).  Outputs: q [numWindows][rowsPerWindow]
 * [cols/2] bytes and scales [numWindows][rowsPerWindow][S] words, q 16-byte
 * and scales 4-byte aligned.  rowCount [numWindows] (device int32, or NULL for
 * all rows): only rows r < rowCount[w] of window w are read and written, as of
 * a dispatch's windows and recvCount.
 * A block's scale byte is clamp(floor(log2 m) + 125, 0, 254), m the block's
 * largest magnitude (0 for a block of zeros); its codes are the elements
 * divided by the scale, to the nearest value, ties to the even code,
 * magnitudes beyond 6 to 6.  A block that holds a NaN or an infinity gets
 * scale byte 255 (NaN) and codes 0.
 */
int epdc_mx_quantize(int32_t numWindows, int32_t rowsPerWindow, int32_t cols, int32_t dtype, const void *x,
                     const int32_t *rowCount, void *q, void *scales, void *stream);

/* The values of quantised rows (epdc_mx_quantize's q, scales and rowCount) as
 * out [numWindows][rowsPerWindow][cols] of outDtype (EPDC_BF16 or EPDC_FP32, 16-byte
 * aligned): code value times scale, exact in both types (infinite past their
 * range, NaN where the scale byte is 255). */
int epdc_mx_dequantize(int32_t numWindows, int32_t rowsPerWindow, int32_t cols, const void *q, const void *scales,
                       const int32_t *rowCount, void *out, int32_t outDtype, void *stream);

/* ------------------------------------------------------------------------
 * Grouping received rows by expert
 * ------------------------------------------------------------------------ */

/* Largest numExpertPerRank of a grouping. */
#define EPDC_MAX_GROUP_EXPERTS 1024

/* Bytes of device scratch epdc_group_experts needs, or 0 if cfg or rank is
 * invalid.  The scratch needs no initial contents; calls that may run at the
 * same time need one each. */
size_t epdc_group_scratch_bytes(const epdc_cfg *cfg, int32_t rank);

/*
 * The (row, slot) pairs of receive windows, sorted by expert.
 *
 * rank in [0, W): the W windows are what PE `rank` received, one window per
 * source, and the Epr experts of that PE are grouped (group e is expert
 * rank*Epr + e; G = Epr groups).  rank = -1: window p is what PE p received
 * from one source, as epdc_dispatch wrote it, and every PE's experts are
 * grouped over its own window (group e is expert e; G = E groups).
 * Inputs (device, read only):
 *   expertIds  [W][M][K] int32: as recvExpertIds
 *   weights    [W][M][K] fp32: as recvWeights; NULL iff useWeights == 0
 *   recvCount  [W] int32 valid rows per window (clamped to [0, M]), or NULL: M each
 * A slot (w, r, k) with r < recvCount[w] whose expert is one of those its
 * window is grouped over is an entry; entries are numbered by expert, then by
 * window, row and slot.
 * Outputs (device):
 *   offsets      [G+1] int32: group e holds entries [offsets[e], offsets[e+1])
 *   entryRow     [W*M*K] int32: the entry's flat row w*M + r
 *   entryWeight  [W*M*K] fp32: its weight; NULL iff useWeights == 0
 *   entryOf      [W][M][K] int32: the slot's entry, -1 for every other slot,
 *                rows past recvCount included.  It is a sendMap into the
 *                entries' rows: epdc_combine with worldSize 1, maxTokPerRank
 *                W*M*K and numTokens W*M sums each row's entries.
 *   entryRow and entryWeight past the last entry are left untouched.
 * hiddenDim, dtype and scaleDim of cfg are not used but checked.
 * EPDC_ERR_INVALID_ARG if W*M*K exceeds 2^31-1 or rank is outside [-1, W);
 * EPDC_ERR_UNSUPPORTED if Epr exceeds EPDC_MAX_GROUP_EXPERTS.
 */
int epdc_group_experts(const epdc_cfg *cfg, int32_t rank, const int32_t *expertIds, const float *weights,
                       const int32_t *recvCount, int32_t *offsets, int32_t *entryRow, float *entryWeight,
                       int32_t *entryOf, void *scratch, size_t scratchBytes, void *stream);

/* ------------------------------------------------------------------------
 * The experts' product
 * ------------------------------------------------------------------------ */

/*
 * out[i] = w_i * (rows[r_i] . weights[e]^T) for every entry i of every group e.
 *
 * numExperts (1..65535) groups of entries, offsets [numExperts+1] int32, ascending: group
 * e holds entries [offsets[e], offsets[e+1]).  (Values are clamped to [0,
 * maxEntries]; where they do not ascend, a group ends at the smallest of the
 * offsets behind its start's, so no entry is in two groups.)
 * rows [numRows][hiddenDim/2] with rowScales [numRows][S] and weights
 * [numExperts][numCols][hiddenDim/2] with weightScales [numExperts][numCols][S]
 * are fp4x2 rows as epdc_mx_quantize makes them (S =
 * epdc_mx_scale_dim(hiddenDim)); hiddenDim counts elements, a multiple of 32.
 * entryRow [maxEntries] int32 is the row r_i of entry i (NULL: r_i = i); an
 * entry whose row is outside [0, numRows) gives a row of +0.
 * entryWeight [maxEntries] fp32 is w_i (NULL: 1).
 * out [maxEntries][numCols] of outDtype (EPDC_BF16 or EPDC_FP32), numCols up
 * to 2^20; its rows must be a multiple of 16 bytes; rows from offsets[numExperts] on (and rows
 * before offsets[0]) are left untouched.
 * Products and sums are fp32 (their order is fixed for given sizes: results
 * are the same from run to run); w_i is applied to the sum, then the result is
 * rounded (nearest, ties to even).  rows, weights and out must be 16-byte
 * aligned, the other arrays 4-byte.
 * maxEntries also chooses the kernel (the groups' sizes are known on the device
 * only): pass the number of entries that can occur, not a far larger capacity,
 * for the best speed -- 64 entries of 32 experts, 7168 -> 4096, take half as
 * long again where maxEntries says 8192.
 */
int epdc_expert_product(int32_t numExperts, int32_t numCols, int32_t hiddenDim, int32_t maxEntries,
                        int32_t numRows, const void *rows, const void *rowScales, const int32_t *offsets,
                        const int32_t *entryRow, const float *entryWeight, const void *weights,
                        const void *weightScales, void *out, int32_t outDtype, void *stream);

/* Message for the last failing call on this thread ("" if none).  The
 * pointer stays valid until the next epdc_* call on the same thread.  MORI
 * JIT v2 design doc, §6: the C entry points report failures through a
 * thread's last-error string rather than exceptions. */
const char *epdc_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* EPDC_H */
