// Host side of the experts in bf16 and int8 (the products grouped by expert
// with their gradients, the gated activation, int8 quantisation): argument
// checks and the launch, in the same manner as epdc_api.cpp -- every check
// runs before anything is enqueued, and no exception escapes.
#include "epdc_host.h"
#include "ops_internal.h"

namespace {

using epdc::host::aligned;
using epdc::host::fail;
using epdc::host::g_lastError;
using epdc::host::hip_status;

bool is_float(int32_t dtype) { return dtype == EPDC_BF16 || dtype == EPDC_FP32; }
int32_t size_of(int32_t dtype) { return dtype == EPDC_FP32 ? 4 : 2; }

int check_type(const char *name, int32_t dtype) {
    if (!is_float(dtype)) return fail(EPDC_ERR_UNSUPPORTED, "%s %d is not EPDC_BF16 or EPDC_FP32", name, dtype);
    return EPDC_OK;
}

int check_groups(int32_t numExperts, int32_t maxEntries) {
    if (numExperts < 1 || numExperts > 65535) return fail(EPDC_ERR_INVALID_ARG, "numExperts %d outside [1, 65535]", numExperts);
    // (a group's length rounded up to whole tiles is an int32)
    if (maxEntries < 0 || maxEntries > EPDC_MAX_EXPERT_ENTRIES)
        return fail(EPDC_ERR_INVALID_ARG, "maxEntries %d outside [0, %d]", maxEntries, EPDC_MAX_EXPERT_ENTRIES);
    return EPDC_OK;
}

// Sizes and types of the products.  colStep and rowStep: what numCols and hiddenDim are multiples of.
int check_product(int32_t numExperts, int32_t numCols, int32_t hiddenDim, int32_t maxEntries, int32_t numRows, int32_t dtype,
                  int32_t colStep, int32_t rowStep) {
    int rc = check_groups(numExperts, maxEntries);
    if (rc == EPDC_OK) rc = check_type("output dtype", dtype);
    if (rc != EPDC_OK) return rc;
    if (hiddenDim < 1 || hiddenDim > EPDC_MAX_EXPERT_DIM)
        return fail(EPDC_ERR_INVALID_ARG, "hiddenDim %d outside [1, %d]", hiddenDim, EPDC_MAX_EXPERT_DIM);
    if (numCols < 1 || numCols > (1 << 20)) return fail(EPDC_ERR_INVALID_ARG, "numCols %d outside [1, %d]", numCols, 1 << 20);
    if (numRows < 0) return fail(EPDC_ERR_INVALID_ARG, "numRows %d < 0", numRows);
    if (hiddenDim % rowStep != 0) return fail(EPDC_ERR_ALIGN, "hiddenDim %d is not a multiple of %d", hiddenDim, rowStep);
    if (numCols % colStep != 0) return fail(EPDC_ERR_ALIGN, "numCols %d is not a multiple of %d", numCols, colStep);
    return EPDC_OK;
}

// Shared by the product and its rows' gradient, after their sizes: pointers, then the parameters.
int product_params(int32_t numExperts, int32_t numCols, int32_t hiddenDim, int32_t maxEntries, int32_t numRows,
                   const void *rows, const int32_t *offsets, const int32_t *entryRow, const float *entryWeight,
                   const void *weights, void *out, epdc::DenseParams &P) {
    if (!offsets || !weights || !out || (numRows > 0 && !rows)) return fail(EPDC_ERR_NULLPTR, "a required product pointer is NULL");
    if (!aligned(rows, 16) || !aligned(weights, 16) || !aligned(out, 16))
        return fail(EPDC_ERR_ALIGN, "rows, weights and the output must be 16-byte aligned");
    if (!aligned(offsets, 4) || !aligned(entryRow, 4) || !aligned(entryWeight, 4))
        return fail(EPDC_ERR_ALIGN, "offsets, entryRow and entryWeight must be 4-byte aligned");
    P.E = numExperts;
    P.N = numCols;
    P.H = hiddenDim;
    P.maxEntries = maxEntries;
    P.numRows = numRows;
    // with no rows every entry is a row of zeros; what is loaded in its place are weights
    P.rows = static_cast<const uint8_t *>(numRows > 0 ? rows : weights);
    P.offsets = offsets;
    P.entryRow = entryRow;
    P.entryWeight = entryWeight;
    P.weights = static_cast<const uint8_t *>(weights);
    P.out = static_cast<uint8_t *>(out);
    return EPDC_OK;
}

int check_gate(int32_t numExperts, int32_t cols, int32_t maxEntries, int32_t dtype, int32_t step) {
    int rc = check_groups(numExperts, maxEntries);
    if (rc == EPDC_OK) rc = check_type("dtype", dtype);
    if (rc != EPDC_OK) return rc;
    if (cols < 1 || cols > EPDC_MAX_EXPERT_DIM)
        return fail(EPDC_ERR_INVALID_ARG, "cols %d outside [1, %d]", cols, EPDC_MAX_EXPERT_DIM);
    if (cols % step != 0) return fail(EPDC_ERR_ALIGN, "cols %d is not a multiple of %d", cols, step);
    return EPDC_OK;
}

int gate_params(int32_t numExperts, int32_t cols, int32_t maxEntries, const void *h, const int32_t *offsets,
                const float *entryWeight, void *out, float *perEntry, epdc::GateParams &P) {
    if (!h || !out) return fail(EPDC_ERR_NULLPTR, "a required gate pointer is NULL");
    if (!aligned(h, 16) || !aligned(out, 16)) return fail(EPDC_ERR_ALIGN, "h and the output must be 16-byte aligned");
    if (!aligned(offsets, 4) || !aligned(entryWeight, 4) || !aligned(perEntry, 4))
        return fail(EPDC_ERR_ALIGN, "int32/fp32 arrays must be 4-byte aligned");
    P.E = numExperts;
    P.F = cols;
    P.maxEntries = maxEntries;
    P.h = static_cast<const uint8_t *>(h);
    P.offsets = offsets;
    P.entryWeight = entryWeight;
    P.out = static_cast<uint8_t *>(out);
    P.perEntry = perEntry;
    return EPDC_OK;
}

}  // namespace

extern "C" {

int epdc_expert_linear(int32_t numExperts, int32_t numCols, int32_t hiddenDim, int32_t maxEntries, int32_t numRows,
                       const void *rows, const int32_t *offsets, const int32_t *entryRow, const float *entryWeight,
                       const void *weights, void *out, int32_t outDtype, void *stream) {
    try {
        g_lastError.clear();
        int rc = check_product(numExperts, numCols, hiddenDim, maxEntries, numRows, outDtype, 16 / size_of(outDtype), 8);
        if (rc != EPDC_OK || maxEntries == 0) return rc;
        epdc::DenseParams P{};
        rc = product_params(numExperts, numCols, hiddenDim, maxEntries, numRows, rows, offsets, entryRow, entryWeight, weights,
                            out, P);
        if (rc != EPDC_OK) return rc;
        const epdc::DenseForm form = epdc::plan_dense(epdc::kDenseProduct, P.E, P.N, P.H, P.maxEntries);
        return hip_status(epdc::launch_dense_linear(P, form, outDtype == EPDC_FP32, static_cast<hipStream_t>(stream)),
                          "bf16 product launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_expert_linear");
    }
}

int epdc_expert_rows_grad(int32_t numExperts, int32_t numCols, int32_t hiddenDim, int32_t maxEntries, int32_t numRows,
                          const void *dOut, const int32_t *offsets, const int32_t *entryRow, const float *entryWeight,
                          const void *weights, void *dRows, int32_t dtype, void *stream) {
    try {
        g_lastError.clear();
        int rc = check_product(numExperts, numCols, hiddenDim, maxEntries, numRows, dtype, 8, 8);
        if (rc != EPDC_OK || maxEntries == 0) return rc;
        epdc::DenseParams P{};
        rc = product_params(numExperts, numCols, hiddenDim, maxEntries, numRows, dOut, offsets, entryRow, entryWeight, weights,
                            dRows, P);
        if (rc != EPDC_OK) return rc;
        const epdc::DenseForm form = epdc::plan_dense(epdc::kDenseRowsGrad, P.E, P.N, P.H, P.maxEntries);
        return hip_status(epdc::launch_dense_rows_grad(P, form, dtype == EPDC_FP32, static_cast<hipStream_t>(stream)),
                          "rows' gradient launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_expert_rows_grad");
    }
}

int epdc_expert_weights_grad(int32_t numExperts, int32_t numCols, int32_t hiddenDim, int32_t maxEntries, int32_t numOutRows,
                             const void *dOut, const int32_t *outRow, int32_t numRows, const void *rows,
                             const int32_t *entryRow, const int32_t *offsets, const void *base, void *dWeights, int32_t dtype,
                             void *stream) {
    try {
        g_lastError.clear();
        const int rc = check_product(numExperts, numCols, hiddenDim, maxEntries, numRows, dtype, 8, 8);
        if (rc != EPDC_OK) return rc;
        if (numOutRows < 0) return fail(EPDC_ERR_INVALID_ARG, "numOutRows %d < 0", numOutRows);
        if (!offsets || !dWeights || (numOutRows > 0 && !dOut) || (numRows > 0 && !rows))
            return fail(EPDC_ERR_NULLPTR, "a required weights' gradient pointer is NULL");
        if (!aligned(dOut, 16) || !aligned(rows, 16) || !aligned(dWeights, 16) || !aligned(base, 16))
            return fail(EPDC_ERR_ALIGN, "dOut, rows, base and dWeights must be 16-byte aligned");
        if (!aligned(offsets, 4) || !aligned(outRow, 4) || !aligned(entryRow, 4))
            return fail(EPDC_ERR_ALIGN, "offsets, outRow and entryRow must be 4-byte aligned");
        epdc::DenseParams P{};
        P.E = numExperts;
        P.N = numCols;
        P.H = hiddenDim;
        // with no rows on a side no entry is one; what is loaded in their place is of the output
        const bool none = numRows == 0 || numOutRows == 0;
        P.maxEntries = none ? 0 : maxEntries;
        P.numRows = numRows;
        P.numOutRows = numOutRows;
        P.rows = static_cast<const uint8_t *>(none ? dWeights : rows);
        P.offsets = offsets;
        P.entryRow = entryRow;
        P.dOut = static_cast<const uint8_t *>(none ? dWeights : dOut);
        P.outRow = outRow;
        P.base = static_cast<const uint8_t *>(base);
        P.out = static_cast<uint8_t *>(dWeights);
        const epdc::DenseForm form = epdc::plan_dense(epdc::kDenseWeightsGrad, P.E, P.N, P.H, P.maxEntries);
        return hip_status(epdc::launch_dense_weights_grad(P, form, dtype == EPDC_FP32, static_cast<hipStream_t>(stream)),
                          "weights' gradient launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_expert_weights_grad");
    }
}

int epdc_expert_linear_int(int32_t numExperts, int32_t numCols, int32_t hiddenDim, int32_t maxEntries, int32_t numRows,
                           const void *rows, const float *rowScales, const int32_t *offsets, const int32_t *entryRow,
                           const float *entryWeight, const void *weights, const float *weightScales, void *out,
                           int32_t outDtype, void *stream) {
    try {
        g_lastError.clear();
        int rc = check_product(numExperts, numCols, hiddenDim, maxEntries, numRows, outDtype, 16 / size_of(outDtype), 16);
        if (rc != EPDC_OK || maxEntries == 0) return rc;
        epdc::DenseParams P{};
        rc = product_params(numExperts, numCols, hiddenDim, maxEntries, numRows, rows, offsets, entryRow, entryWeight, weights,
                            out, P);
        if (rc != EPDC_OK) return rc;
        if (!weightScales || (numRows > 0 && !rowScales)) return fail(EPDC_ERR_NULLPTR, "rowScales or weightScales is NULL");
        if (!aligned(rowScales, 4) || !aligned(weightScales, 4))
            return fail(EPDC_ERR_ALIGN, "rowScales and weightScales must be 4-byte aligned");
        P.rowScales = rowScales;
        P.weightScales = weightScales;
        const epdc::DenseForm form = epdc::plan_dense(epdc::kDenseProduct, P.E, P.N, P.H, P.maxEntries);
        return hip_status(epdc::launch_dense_linear_int(P, form, outDtype == EPDC_FP32, static_cast<hipStream_t>(stream)),
                          "int8 product launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_expert_linear_int");
    }
}

int epdc_expert_gate(int32_t numExperts, int32_t cols, int32_t maxEntries, int32_t dtype, const void *h,
                     const int32_t *offsets, const float *entryWeight, void *out, int32_t outDtype, void *stream) {
    try {
        g_lastError.clear();
        int rc = check_gate(numExperts, cols, maxEntries, dtype, 8);
        if (rc == EPDC_OK) rc = check_type("outDtype", outDtype);
        if (rc != EPDC_OK || maxEntries == 0) return rc;
        epdc::GateParams P{};
        rc = gate_params(numExperts, cols, maxEntries, h, offsets, entryWeight, out, nullptr, P);
        if (rc != EPDC_OK) return rc;
        return hip_status(epdc::launch_gate(P, dtype == EPDC_FP32, outDtype == EPDC_FP32, static_cast<hipStream_t>(stream)),
                          "gate launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_expert_gate");
    }
}

int epdc_expert_gate_grad(int32_t numExperts, int32_t cols, int32_t maxEntries, int32_t dtype, const void *h,
                          const int32_t *offsets, const float *entryWeight, const void *dOut, int32_t outDtype, void *dH,
                          float *dEntryWeight, void *stream) {
    try {
        g_lastError.clear();
        int rc = check_gate(numExperts, cols, maxEntries, dtype, 8);
        if (rc == EPDC_OK) rc = check_type("outDtype", outDtype);
        if (rc != EPDC_OK || maxEntries == 0) return rc;
        epdc::GateParams P{};
        rc = gate_params(numExperts, cols, maxEntries, h, offsets, entryWeight, dH, dEntryWeight, P);
        if (rc != EPDC_OK) return rc;
        if (!dOut) return fail(EPDC_ERR_NULLPTR, "dOut is NULL");
        if (!aligned(dOut, 16)) return fail(EPDC_ERR_ALIGN, "dOut must be 16-byte aligned");
        P.dOut = static_cast<const uint8_t *>(dOut);
        return hip_status(epdc::launch_gate_grad(P, dtype == EPDC_FP32, outDtype == EPDC_FP32, static_cast<hipStream_t>(stream)),
                          "gate gradient launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_expert_gate_grad");
    }
}

int epdc_expert_gate_int(int32_t numExperts, int32_t cols, int32_t maxEntries, int32_t dtype, const void *h,
                         const int32_t *offsets, const float *entryWeight, void *q, float *scales, void *stream) {
    try {
        g_lastError.clear();
        int rc = check_gate(numExperts, cols, maxEntries, dtype, 16);
        if (rc != EPDC_OK || maxEntries == 0) return rc;
        epdc::GateParams P{};
        rc = gate_params(numExperts, cols, maxEntries, h, offsets, entryWeight, q, scales, P);
        if (rc != EPDC_OK) return rc;
        if (!scales) return fail(EPDC_ERR_NULLPTR, "scales is NULL");
        return hip_status(epdc::launch_gate_int(P, dtype == EPDC_FP32, static_cast<hipStream_t>(stream)), "int8 gate launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_expert_gate_int");
    }
}

int epdc_int_quantize(int32_t numWindows, int32_t rowsPerWindow, int32_t cols, int32_t dtype, const void *x,
                      const int32_t *rowCount, void *q, float *scales, void *stream) {
    try {
        g_lastError.clear();
        if (numWindows < 0 || rowsPerWindow < 0)
            return fail(EPDC_ERR_INVALID_ARG, "numWindows %d or rowsPerWindow %d < 0", numWindows, rowsPerWindow);
        if ((int64_t)numWindows * rowsPerWindow > INT32_MAX)
            return fail(EPDC_ERR_INVALID_ARG, "numWindows*rowsPerWindow overflows int32");
        if (cols < 1 || cols > EPDC_MAX_EXPERT_DIM)
            return fail(EPDC_ERR_INVALID_ARG, "cols %d outside [1, %d]", cols, EPDC_MAX_EXPERT_DIM);
        if (cols % 16 != 0) return fail(EPDC_ERR_ALIGN, "cols %d is not a multiple of 16", cols);
        const int rc = check_type("dtype", dtype);
        if (rc != EPDC_OK) return rc;
        if (!aligned(rowCount, 4)) return fail(EPDC_ERR_ALIGN, "rowCount must be 4-byte aligned");
        epdc::Int8Params P{};
        P.rows = (int64_t)numWindows * rowsPerWindow;
        if (P.rows == 0) return EPDC_OK;
        if (!x || !q || !scales) return fail(EPDC_ERR_NULLPTR, "a required quantise pointer is NULL");
        if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 4))
            return fail(EPDC_ERR_ALIGN, "x and q must be 16-byte aligned, scales 4-byte");
        P.M = rowsPerWindow;
        P.cols = cols;
        P.rowCount = rowCount;
        P.x = static_cast<const uint8_t *>(x);
        P.q = static_cast<uint8_t *>(q);
        P.scales = scales;
        return hip_status(epdc::launch_int_quantize(P, dtype == EPDC_FP32, static_cast<hipStream_t>(stream)),
                          "int8 quantise launch");
    } catch (...) {
        return fail(EPDC_ERR_HIP, "unexpected C++ exception in epdc_int_quantize");
    }
}

}  // extern "C"
