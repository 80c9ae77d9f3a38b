// Host side of the entry points next to dispatch and combine (routing, fp4x2
// quantisation, grouping by expert, the experts' product): argument checks
// and the launch, in the same manner as epdc_api.cpp -- every check runs
// before anything is enqueued, and no exception escapes.
#include <cmath>

#include "epdc_host.h"
#include "ops_internal.h"

namespace {

using epdc::host::aligned;
using epdc::host::check_cfg;
using epdc::host::fail;
using epdc::host::g_lastError;
using epdc::host::hip_status;

int check_route_cfg(const epdc_route_cfg *c, int32_t numTokens) {
    if (!c) return fail(EPDC_ERR_NULLPTR, "cfg is NULL");
    if (c->numExperts < 1 || c->numExperts > EPDC_MAX_ROUTE_EXPERTS)
        return fail(EPDC_ERR_INVALID_ARG, "numExperts %d outside [1, %d]", c->numExperts, EPDC_MAX_ROUTE_EXPERTS);
    if (c->numExpertPerToken < 1 || c->numExpertPerToken > 64)
        return fail(EPDC_ERR_INVALID_ARG, "numExpertPerToken %d outside [1, 64]", c->numExpertPerToken);
    if (c->dtype != EPDC_BF16 && c->dtype != EPDC_FP32)
        return fail(EPDC_ERR_UNSUPPORTED, "logits' dtype %d is not EPDC_BF16 or EPDC_FP32", c->dtype);
    if (c->score != EPDC_SOFTMAX && c->score != EPDC_SIGMOID)
        return fail(EPDC_ERR_UNSUPPORTED, "score %d is not EPDC_SOFTMAX or EPDC_SIGMOID", c->score);
    if (c->numGroups < 1 || c->numGroups > 64 || c->numExperts % c->numGroups != 0)
        return fail(EPDC_ERR_INVALID_ARG, "numGroups %d outside [1, 64] or not a divisor of numExperts %d", c->numGroups,
                    c->numExperts);
    const int32_t perGroup = c->numExperts / c->numGroups;
    if (c->groupsPerToken < 1 || c->groupsPerToken > c->numGroups)
        return fail(EPDC_ERR_INVALID_ARG, "groupsPerToken %d outside [1, numGroups %d]", c->groupsPerToken, c->numGroups);
    if (c->groupTop < 1 || c->groupTop > 2 || c->groupTop > perGroup)
        return fail(EPDC_ERR_INVALID_ARG, "groupTop %d is not 1 or 2, or above the %d experts of a group", c->groupTop,
                    perGroup);
    if (c->numExpertPerToken > c->groupsPerToken * perGroup)
        return fail(EPDC_ERR_INVALID_ARG, "numExpertPerToken %d > %d experts of groupsPerToken groups",
                    c->numExpertPerToken, c->groupsPerToken * perGroup);
    if (c->renormalize != 0 && c->renormalize != 1)
        return fail(EPDC_ERR_UNSUPPORTED, "renormalize must be 0 or 1, got %d", c->renormalize);
    if (!std::isfinite(c->routedScale)) return fail(EPDC_ERR_INVALID_ARG, "routedScale is not finite");
    if (numTokens < 0) return fail(EPDC_ERR_INVALID_ARG, "numTokens %d < 0", numTokens);
    return EPDC_OK;
}

// Logit arrays are read element by element where they are not 16-byte
// aligned: only the element's own alignment is asked for.
bool logits_aligned(const epdc_route_cfg *c, const void *p) { return aligned(p, c->dtype == EPDC_FP32 ? 4 : 2); }

int32_t scale_dim(int32_t cols) {
    if (cols < 32 || cols % 32 != 0 || cols > 128 * EPDC_MAX_SCALE_DIM) return -1;
    return (cols + 127) / 128;
}

// Shape checks and parameters shared by quantise and dequantise.
int mx_params(int32_t numWindows, int32_t rowsPerWindow, int32_t cols, int32_t dtype, const int32_t *rowCount,
              epdc::MxParams &P) {
    if (numWindows < 0 || rowsPerWindow < 0)
        return fail(EPDC_ERR_INVALID_ARG, "numWindows %d or rowsPerWindow %d < 0", numWindows, rowsPerWindow);
    if ((int64_t)numWindows * rowsPerWindow > INT32_MAX)
        return fail(EPDC_ERR_INVALID_ARG, "numWindows*rowsPerWindow overflows int32");
    if (scale_dim(cols) < 0)
        return fail(EPDC_ERR_INVALID_ARG, "cols %d is not a multiple of 32 in [32, %d]", cols, 128 * EPDC_MAX_SCALE_DIM);
    if (dtype != EPDC_BF16 && dtype != EPDC_FP32)
        return fail(EPDC_ERR_UNSUPPORTED, "dtype %d is not EPDC_BF16 or EPDC_FP32", dtype);
    if (!aligned(rowCount, 4)) return fail(EPDC_ERR_ALIGN, "rowCount must be 4-byte aligned");
    P.units = (int64_t)numWindows * rowsPerWindow * (cols / 8);
    P.unitsPerRow = cols / 8;
    P.M = rowsPerWindow;
    P.words = scale_dim(cols);
    P.rowDiv = epdc::div_magic((uint32_t)P.unitsPerRow);
    P.winDiv = epdc::div_magic((uint32_t)(rowsPerWindow > 0 ? rowsPerWindow : 1));
    P.rowCount = rowCount;
    return EPDC_OK;
}

int check_group(const epdc_cfg *cfg, int32_t rank) {
    const int rc = check_cfg(cfg, 0, false);
    if (rc != EPDC_OK) return rc;
    if (rank < -1 || rank >= cfg->worldSize)
        return fail(EPDC_ERR_INVALID_ARG, "rank %d outside [-1, worldSize %d)", rank, cfg->worldSize);
    if ((int64_t)cfg->worldSize * cfg->maxTokPerRank * cfg->numExpertPerToken > INT32_MAX)
        return fail(EPDC_ERR_INVALID_ARG, "worldSize*maxTokPerRank*numExpertPerToken overflows int32");
    if (cfg->numExpertPerRank > EPDC_MAX_GROUP_EXPERTS)
        return fail(EPDC_ERR_UNSUPPORTED, "numExpertPerRank %d > %d", cfg->numExpertPerRank, EPDC_MAX_GROUP_EXPERTS);
    return EPDC_OK;
}

size_t group_bytes(const epdc_cfg *c) {
    return (size_t)epdc::group_scratch_words(c->worldSize, c->maxTokPerRank, c->numExpertPerToken, c->numExpertPerRank) *
           sizeof(int32_t);
}

}  // namespace

extern "C" {

int epdc_route(const epdc_route_cfg *cfg, int32_t numTokens, const void *logits, const float *bias, int32_t *expertIds,
               float *weights, void *stream) {
    try {
        g_lastError.clear();
        const int rc = check_route_cfg(cfg, numTokens);
        if (rc != EPDC_OK) return rc;
        if (numTokens == 0) return EPDC_OK;
        if (!logits || !expertIds || !weights) return fail(EPDC_ERR_NULLPTR, "a required route pointer is NULL");
        if (!logits_aligned(cfg, logits)) return fail(EPDC_ERR_ALIGN, "logits must be aligned to their element");
        if (!aligned(bias, 4) || !aligned(expertIds, 4) || !aligned(weights, 4))
            return fail(EPDC_ERR_ALIGN, "int32/fp32 arrays must be 4-byte aligned");
        epdc::RouteParams P{};
        P.E = cfg->numExperts;
        P.K = cfg->numExpertPerToken;
        P.T = numTokens;
        P.G = cfg->numGroups;
        P.keep = cfg->groupsPerToken;
        P.groupTop = cfg->groupTop;
        P.perGroup = cfg->numExperts / cfg->numGroups;
        P.softmax = cfg->score == EPDC_SOFTMAX;
        P.renorm = cfg->renormalize;
        P.scale = cfg->routedScale;
        P.logits = logits;
        P.bias = bias;
        P.expertIds = expertIds;
        P.weights = weights;
        return hip_status(epdc::launch_route(P, cfg->dtype == EPDC_FP32, static_cast<hipStream_t>(stream)), "route launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_route");
    }
}

int epdc_route_grad(const epdc_route_cfg *cfg, int32_t numTokens, const void *logits, const int32_t *expertIds,
                    const float *dWeights, void *dLogits, void *stream) {
    try {
        g_lastError.clear();
        const int rc = check_route_cfg(cfg, numTokens);
        if (rc != EPDC_OK) return rc;
        if (numTokens == 0) return EPDC_OK;
        if (!logits || !expertIds || !dWeights || !dLogits)
            return fail(EPDC_ERR_NULLPTR, "a required route gradient pointer is NULL");
        if (!logits_aligned(cfg, logits) || !logits_aligned(cfg, dLogits))
            return fail(EPDC_ERR_ALIGN, "logits and dLogits must be aligned to their element");
        if (!aligned(expertIds, 4) || !aligned(dWeights, 4))
            return fail(EPDC_ERR_ALIGN, "int32/fp32 arrays must be 4-byte aligned");
        epdc::RouteGradParams P{};
        P.E = cfg->numExperts;
        P.K = cfg->numExpertPerToken;
        P.T = numTokens;
        P.softmax = cfg->score == EPDC_SOFTMAX;
        P.renorm = cfg->renormalize;
        P.scale = cfg->routedScale;
        P.logits = logits;
        P.expertIds = expertIds;
        P.dWeights = dWeights;
        P.dLogits = dLogits;
        return hip_status(epdc::launch_route_grad(P, cfg->dtype == EPDC_FP32, static_cast<hipStream_t>(stream)),
                          "route gradient launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_route_grad");
    }
}

int32_t epdc_mx_scale_dim(int32_t cols) { return scale_dim(cols); }

int epdc_mx_quantize(int32_t numWindows, int32_t rowsPerWindow, int32_t cols, int32_t dtype, const void *x,
                     const int32_t *rowCount, void *q, void *scales, void *stream) {
    try {
        g_lastError.clear();
        epdc::MxParams P{};
        const int rc = mx_params(numWindows, rowsPerWindow, cols, dtype, rowCount, P);
        if (rc != EPDC_OK) return rc;
        if (P.units == 0) return EPDC_OK;
        if (!x || !q || !scales) return fail(EPDC_ERR_NULLPTR, "a required quantise pointer is NULL");
        if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 4))
            return fail(EPDC_ERR_ALIGN, "x and q must be 16-byte aligned, scales 4-byte");
        P.in = static_cast<const uint8_t *>(x);
        P.out = static_cast<uint8_t *>(q);
        P.scales = static_cast<uint8_t *>(scales);
        return hip_status(epdc::launch_mx_quantize(P, dtype == EPDC_FP32, static_cast<hipStream_t>(stream)), "quantise launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_mx_quantize");
    }
}

int epdc_mx_dequantize(int32_t numWindows, int32_t rowsPerWindow, int32_t cols, const void *q, const void *scales,
                       const int32_t *rowCount, void *out, int32_t outDtype, void *stream) {
    try {
        g_lastError.clear();
        epdc::MxParams P{};
        const int rc = mx_params(numWindows, rowsPerWindow, cols, outDtype, rowCount, P);
        if (rc != EPDC_OK) return rc;
        if (P.units == 0) return EPDC_OK;
        if (!q || !scales || !out) return fail(EPDC_ERR_NULLPTR, "a required dequantise pointer is NULL");
        if (!aligned(q, 16) || !aligned(out, 16) || !aligned(scales, 4))
            return fail(EPDC_ERR_ALIGN, "q and out must be 16-byte aligned, scales 4-byte");
        P.in = static_cast<const uint8_t *>(q);
        P.out = static_cast<uint8_t *>(out);
        P.scales = const_cast<uint8_t *>(static_cast<const uint8_t *>(scales));
        return hip_status(epdc::launch_mx_dequantize(P, outDtype == EPDC_FP32, static_cast<hipStream_t>(stream)),
                          "dequantise launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_mx_dequantize");
    }
}

size_t epdc_group_scratch_bytes(const epdc_cfg *cfg, int32_t rank) {
    try {
        if (check_group(cfg, rank) != EPDC_OK) return 0;
        return group_bytes(cfg);
    } catch (...) {
        return 0;
    }
}

int epdc_group_experts(const epdc_cfg *cfg, int32_t rank, const int32_t *expertIds, const float *weights,
                       const int32_t *recvCount, int32_t *offsets, int32_t *entryRow, float *entryWeight,
                       int32_t *entryOf, void *scratch, size_t scratchBytes, void *stream) {
    try {
        g_lastError.clear();
        const int rc = check_group(cfg, rank);
        if (rc != EPDC_OK) return rc;
        if (!expertIds || !offsets || !entryRow || !entryOf) return fail(EPDC_ERR_NULLPTR, "a required group pointer is NULL");
        if (cfg->useWeights && (!weights || !entryWeight))
            return fail(EPDC_ERR_NULLPTR, "useWeights=1 needs weights and entryWeight");
        if (!scratch) return fail(EPDC_ERR_NULLPTR, "scratch is NULL");
        if (!aligned(expertIds, 4) || !aligned(recvCount, 4) || !aligned(offsets, 4) || !aligned(entryRow, 4) ||
            !aligned(entryOf, 4) || (cfg->useWeights && (!aligned(weights, 4) || !aligned(entryWeight, 4))))
            return fail(EPDC_ERR_ALIGN, "int32/fp32 arrays must be 4-byte aligned");
        if (!aligned(scratch, 16)) return fail(EPDC_ERR_ALIGN, "scratch must be 16-byte aligned");
        if (scratchBytes < group_bytes(cfg))
            return fail(EPDC_ERR_SCRATCH, "scratchBytes %zu < %zu required", scratchBytes, group_bytes(cfg));
        epdc::GroupParams P{};
        P.W = cfg->worldSize;
        P.M = cfg->maxTokPerRank;
        P.K = cfg->numExpertPerToken;
        P.Epr = cfg->numExpertPerRank;
        P.rank = rank;
        P.tileRows = epdc::group_tile_rows(P.K);
        P.tilesPerWindow = epdc::group_tiles_per_window(P.M, P.K);
        P.windowDiv = epdc::div_magic((uint32_t)P.M * (uint32_t)P.K);
        P.expertIds = expertIds;
        P.weights = cfg->useWeights ? weights : nullptr;
        P.recvCount = recvCount;
        P.offsets = offsets;
        P.entryRow = entryRow;
        P.entryWeight = cfg->useWeights ? entryWeight : nullptr;
        P.entryOf = entryOf;
        P.hist = static_cast<int32_t *>(scratch);
        return hip_status(epdc::launch_group(P, static_cast<hipStream_t>(stream)), "group launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_group_experts");
    }
}

int epdc_expert_product(int32_t numExperts, int32_t numCols, int32_t hiddenDim, int32_t maxEntries, int32_t numRows,
                        const void *rows, const void *rowScales, const int32_t *offsets, const int32_t *entryRow,
                        const float *entryWeight, const void *weights, const void *weightScales, void *out,
                        int32_t outDtype, void *stream) {
    try {
        g_lastError.clear();
        if (numExperts < 1 || numExperts > 65535) return fail(EPDC_ERR_INVALID_ARG, "numExperts %d outside [1, 65535]", numExperts);
        if (scale_dim(hiddenDim) < 0)
            return fail(EPDC_ERR_INVALID_ARG, "hiddenDim %d is not a multiple of 32 in [32, %d]", hiddenDim,
                        128 * EPDC_MAX_SCALE_DIM);
        if (outDtype != EPDC_BF16 && outDtype != EPDC_FP32)
            return fail(EPDC_ERR_UNSUPPORTED, "outDtype %d is not EPDC_BF16 or EPDC_FP32", outDtype);
        const int32_t ob = outDtype == EPDC_FP32 ? 4 : 2;
        if (numCols < 1 || numCols > (1 << 20)) return fail(EPDC_ERR_INVALID_ARG, "numCols %d outside [1, %d]", numCols, 1 << 20);
        if ((numCols * ob) % 16 != 0)
            return fail(EPDC_ERR_ALIGN, "output row of %d bytes is not a multiple of 16", numCols * ob);
        if (maxEntries < 0 || numRows < 0)
            return fail(EPDC_ERR_INVALID_ARG, "maxEntries %d or numRows %d < 0", maxEntries, numRows);
        if (maxEntries == 0) return EPDC_OK;
        if (!offsets || !weights || !weightScales || !out || (numRows > 0 && (!rows || !rowScales)))
            return fail(EPDC_ERR_NULLPTR, "a required product pointer is NULL");
        if (!aligned(rows, 16) || !aligned(weights, 16) || !aligned(out, 16))
            return fail(EPDC_ERR_ALIGN, "rows, weights and out must be 16-byte aligned");
        if (!aligned(rowScales, 4) || !aligned(weightScales, 4) || !aligned(offsets, 4) || !aligned(entryRow, 4) ||
            !aligned(entryWeight, 4))
            return fail(EPDC_ERR_ALIGN, "scales, offsets, entryRow and entryWeight must be 4-byte aligned");
        epdc::ProductParams P{};
        P.E = numExperts;
        P.N = numCols;
        P.H = hiddenDim;
        P.maxEntries = maxEntries;
        P.numRows = numRows;
        P.rowBytes = hiddenDim / 2;
        P.words = scale_dim(hiddenDim);
        // with no rows every entry is a row of zeros; what is loaded in its place is a weight row
        P.rows = static_cast<const uint8_t *>(numRows > 0 ? rows : weights);
        P.rowScales = static_cast<const uint8_t *>(numRows > 0 ? rowScales : weightScales);
        P.offsets = offsets;
        P.entryRow = entryRow;
        P.entryWeight = entryWeight;
        P.weights = static_cast<const uint8_t *>(weights);
        P.weightScales = static_cast<const uint8_t *>(weightScales);
        P.out = out;
        return hip_status(epdc::launch_product(P, outDtype == EPDC_FP32, static_cast<hipStream_t>(stream)), "product launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_expert_product");
    }
}

}  // extern "C"
