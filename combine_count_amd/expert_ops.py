"""Binding of the experts in bf16 and int8 (include/epdc.h, last part): the
products grouped by expert with their gradients, the gated activation between
them with its gradient, and the int8 form with a scale per token and column.

The same manner as layer_ops.py: argument marshalling only, the same checks of
tensors, a prepare_* form of every call.
"""
from __future__ import annotations

from .binding import PreparedCall
from .layer_ops import _BYTES, _FLOATS, _array, _call, _i

_F, _I, _B = "torch.float32", "torch.int32", "torch.bfloat16"
_CODES = "torch.int8"


def _sizes(*values):
    return tuple(max(int(v), 0) for v in values)


def prepare_expert_linear(numExperts: int, numCols: int, hiddenDim: int, maxEntries: int, numRows: int, rows, offsets,
                          entryRow, entryWeight, weights, out, outDtype: int) -> PreparedCall:
    E, N, H, n, R = _sizes(numExperts, numCols, hiddenDim, maxEntries, numRows)
    args = [_i(numExperts), _i(numCols), _i(hiddenDim), _i(maxEntries), _i(numRows), _array(rows, R * H * 2, "rows", _B),
            _array(offsets, (E + 1) * 4, "offsets", _I), _array(entryRow, n * 4, "entryRow", _I),
            _array(entryWeight, n * 4, "entryWeight", _F), _array(weights, E * N * H * 2, "weights", _B),
            _array(out, n * N * _BYTES.get(outDtype, 0), "out", _FLOATS.get(outDtype)), _i(outDtype)]
    return _call("epdc_expert_linear", args, (rows, offsets, entryRow, entryWeight, weights, out))


def prepare_expert_rows_grad(numExperts: int, numCols: int, hiddenDim: int, maxEntries: int, numRows: int, dOut, offsets,
                             entryRow, entryWeight, weights, dRows, dtype: int) -> PreparedCall:
    E, N, H, n, R = _sizes(numExperts, numCols, hiddenDim, maxEntries, numRows)
    args = [_i(numExperts), _i(numCols), _i(hiddenDim), _i(maxEntries), _i(numRows), _array(dOut, R * N * 2, "dOut", _B),
            _array(offsets, (E + 1) * 4, "offsets", _I), _array(entryRow, n * 4, "entryRow", _I),
            _array(entryWeight, n * 4, "entryWeight", _F), _array(weights, E * N * H * 2, "weights", _B),
            _array(dRows, n * H * _BYTES.get(dtype, 0), "dRows", _FLOATS.get(dtype)), _i(dtype)]
    return _call("epdc_expert_rows_grad", args, (dOut, offsets, entryRow, entryWeight, weights, dRows))


def prepare_expert_weights_grad(numExperts: int, numCols: int, hiddenDim: int, maxEntries: int, numOutRows: int, dOut, outRow,
                                numRows: int, rows, entryRow, offsets, base, dWeights, dtype: int) -> PreparedCall:
    E, N, H, n, D, R = _sizes(numExperts, numCols, hiddenDim, maxEntries, numOutRows, numRows)
    whole, kind = E * N * H * _BYTES.get(dtype, 0), _FLOATS.get(dtype)
    args = [_i(numExperts), _i(numCols), _i(hiddenDim), _i(maxEntries), _i(numOutRows), _array(dOut, D * N * 2, "dOut", _B),
            _array(outRow, n * 4, "outRow", _I), _i(numRows), _array(rows, R * H * 2, "rows", _B),
            _array(entryRow, n * 4, "entryRow", _I), _array(offsets, (E + 1) * 4, "offsets", _I),
            _array(base, whole, "base", kind), _array(dWeights, whole, "dWeights", kind), _i(dtype)]
    return _call("epdc_expert_weights_grad", args, (dOut, outRow, rows, entryRow, offsets, base, dWeights))


def prepare_expert_gate(numExperts: int, cols: int, maxEntries: int, dtype: int, h, offsets, entryWeight, out,
                        outDtype: int) -> PreparedCall:
    E, F, n = _sizes(numExperts, cols, maxEntries)
    args = [_i(numExperts), _i(cols), _i(maxEntries), _i(dtype),
            _array(h, n * 2 * F * _BYTES.get(dtype, 0), "h", _FLOATS.get(dtype)),
            _array(offsets, (E + 1) * 4, "offsets", _I), _array(entryWeight, n * 4, "entryWeight", _F),
            _array(out, n * F * _BYTES.get(outDtype, 0), "out", _FLOATS.get(outDtype)), _i(outDtype)]
    return _call("epdc_expert_gate", args, (h, offsets, entryWeight, out))


def prepare_expert_gate_grad(numExperts: int, cols: int, maxEntries: int, dtype: int, h, offsets, entryWeight, dOut,
                             outDtype: int, dH, dEntryWeight) -> PreparedCall:
    E, F, n = _sizes(numExperts, cols, maxEntries)
    whole, kind = n * 2 * F * _BYTES.get(dtype, 0), _FLOATS.get(dtype)
    args = [_i(numExperts), _i(cols), _i(maxEntries), _i(dtype), _array(h, whole, "h", kind),
            _array(offsets, (E + 1) * 4, "offsets", _I), _array(entryWeight, n * 4, "entryWeight", _F),
            _array(dOut, n * F * _BYTES.get(outDtype, 0), "dOut", _FLOATS.get(outDtype)), _i(outDtype),
            _array(dH, whole, "dH", kind), _array(dEntryWeight, n * 4, "dEntryWeight", _F)]
    return _call("epdc_expert_gate_grad", args, (h, offsets, entryWeight, dOut, dH, dEntryWeight))


def prepare_int_quantize(numWindows: int, rowsPerWindow: int, cols: int, dtype: int, x, rowCount, q, scales) -> PreparedCall:
    W, M, C = _sizes(numWindows, rowsPerWindow, cols)
    args = [_i(numWindows), _i(rowsPerWindow), _i(cols), _i(dtype),
            _array(x, W * M * C * _BYTES.get(dtype, 0), "x", _FLOATS.get(dtype)), _array(rowCount, W * 4, "rowCount", _I),
            _array(q, W * M * C, "q", size=1), _array(scales, W * M * 4, "scales", _F)]
    return _call("epdc_int_quantize", args, (x, rowCount, q, scales))


def prepare_expert_gate_int(numExperts: int, cols: int, maxEntries: int, dtype: int, h, offsets, entryWeight, q,
                            scales) -> PreparedCall:
    E, F, n = _sizes(numExperts, cols, maxEntries)
    args = [_i(numExperts), _i(cols), _i(maxEntries), _i(dtype),
            _array(h, n * 2 * F * _BYTES.get(dtype, 0), "h", _FLOATS.get(dtype)),
            _array(offsets, (E + 1) * 4, "offsets", _I), _array(entryWeight, n * 4, "entryWeight", _F),
            _array(q, n * F, "q", size=1), _array(scales, n * 4, "scales", _F)]
    return _call("epdc_expert_gate_int", args, (h, offsets, entryWeight, q, scales))


def prepare_expert_linear_int(numExperts: int, numCols: int, hiddenDim: int, maxEntries: int, numRows: int, rows, rowScales,
                              offsets, entryRow, entryWeight, weights, weightScales, out, outDtype: int) -> PreparedCall:
    E, N, H, n, R = _sizes(numExperts, numCols, hiddenDim, maxEntries, numRows)
    args = [_i(numExperts), _i(numCols), _i(hiddenDim), _i(maxEntries), _i(numRows), _array(rows, R * H, "rows", size=1),
            _array(rowScales, R * 4, "rowScales", _F), _array(offsets, (E + 1) * 4, "offsets", _I),
            _array(entryRow, n * 4, "entryRow", _I), _array(entryWeight, n * 4, "entryWeight", _F),
            _array(weights, E * N * H, "weights", _CODES), _array(weightScales, E * N * 4, "weightScales", _F),
            _array(out, n * N * _BYTES.get(outDtype, 0), "out", _FLOATS.get(outDtype)), _i(outDtype)]
    return _call("epdc_expert_linear_int", args,
                 (rows, rowScales, offsets, entryRow, entryWeight, weights, weightScales, out))


def epdc_expert_linear(numExperts: int, numCols: int, hiddenDim: int, maxEntries: int, numRows: int, rows, offsets,
                       entryRow, entryWeight, weights, out, outDtype: int, stream=None, check: bool = True) -> int:
    return prepare_expert_linear(numExperts, numCols, hiddenDim, maxEntries, numRows, rows, offsets, entryRow,
                                 entryWeight, weights, out, outDtype)(stream, check)


def epdc_expert_rows_grad(numExperts: int, numCols: int, hiddenDim: int, maxEntries: int, numRows: int, dOut, offsets, entryRow,
                          entryWeight, weights, dRows, dtype: int, stream=None, check: bool = True) -> int:
    return prepare_expert_rows_grad(numExperts, numCols, hiddenDim, maxEntries, numRows, dOut, offsets, entryRow, entryWeight,
                                    weights, dRows, dtype)(stream, check)


def epdc_expert_weights_grad(numExperts: int, numCols: int, hiddenDim: int, maxEntries: int, numOutRows: int, dOut, outRow,
                             numRows: int, rows, entryRow, offsets, base, dWeights, dtype: int, stream=None,
                             check: bool = True) -> int:
    return prepare_expert_weights_grad(numExperts, numCols, hiddenDim, maxEntries, numOutRows, dOut, outRow, numRows, rows,
                                       entryRow, offsets, base, dWeights, dtype)(stream, check)


def epdc_expert_gate(numExperts: int, cols: int, maxEntries: int, dtype: int, h, offsets, entryWeight, out, outDtype: int,
                     stream=None, check: bool = True) -> int:
    return prepare_expert_gate(numExperts, cols, maxEntries, dtype, h, offsets, entryWeight, out, outDtype)(stream, check)


def epdc_expert_gate_grad(numExperts: int, cols: int, maxEntries: int, dtype: int, h, offsets, entryWeight, dOut, outDtype: int,
                          dH, dEntryWeight, stream=None, check: bool = True) -> int:
    return prepare_expert_gate_grad(numExperts, cols, maxEntries, dtype, h, offsets, entryWeight, dOut, outDtype, dH,
                                    dEntryWeight)(stream, check)


def epdc_int_quantize(numWindows: int, rowsPerWindow: int, cols: int, dtype: int, x, rowCount, q, scales, stream=None,
                      check: bool = True) -> int:
    return prepare_int_quantize(numWindows, rowsPerWindow, cols, dtype, x, rowCount, q, scales)(stream, check)


def epdc_expert_gate_int(numExperts: int, cols: int, maxEntries: int, dtype: int, h, offsets, entryWeight, q, scales,
                         stream=None, check: bool = True) -> int:
    return prepare_expert_gate_int(numExperts, cols, maxEntries, dtype, h, offsets, entryWeight, q, scales)(stream, check)


def epdc_expert_linear_int(numExperts: int, numCols: int, hiddenDim: int, maxEntries: int, numRows: int, rows, rowScales,
                           offsets, entryRow, entryWeight, weights, weightScales, out, outDtype: int, stream=None,
                           check: bool = True) -> int:
    return prepare_expert_linear_int(numExperts, numCols, hiddenDim, maxEntries, numRows, rows, rowScales, offsets, entryRow,
                                     entryWeight, weights, weightScales, out, outDtype)(stream, check)
