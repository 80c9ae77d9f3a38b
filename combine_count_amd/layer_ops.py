"""Binding of the operators next to dispatch and combine (include/epdc.h):
routing and its gradient, fp4x2 quantisation, grouping of received rows by
expert, and the experts' product.

The same manner as binding.py: argument marshalling only.  Tensors must be on
the current device, contiguous, of the element type the header states and at
least as large as the call needs, or a ValueError is raised before anything
is launched; a negative return code becomes an EpdcError.  Every call has a
prepare_* form that marshals its arguments once (PreparedCall).
"""
from __future__ import annotations

import ctypes

from . import binding as _b
from .binding import EPDC_BF16, EPDC_FP32, EpCfg, PreparedCall, RouteCfg, load_library

_FLOATS = {EPDC_BF16: "torch.bfloat16", EPDC_FP32: "torch.float32"}
_BYTES = {EPDC_BF16: 2, EPDC_FP32: 4}


def _array(a, nbytes: int, name: str, kind=None, size: int = 0):
    """Device address of an array argument (None and raw addresses as they
    are) after its checks: on the current device, contiguous, of dtype `kind`
    (or of `size`-byte elements), at least `nbytes` long."""
    if a is None:
        return None
    if isinstance(a, int):
        return ctypes.c_void_p(a)
    addr = _b._ptr(a)
    import torch
    if a.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {a.device}, the current device is cuda:{torch.cuda.current_device()}")
    if kind is not None and str(a.dtype) != kind:
        raise ValueError(f"{name} must be {kind}, got {a.dtype}")
    if size and a.element_size() != size:
        raise ValueError(f"{name} must have {size}-byte elements, got {a.dtype}")
    _b._need(a, nbytes, name)
    return ctypes.c_void_p(addr)


def _call(name: str, args, keep):
    return PreparedCall(getattr(_b._lib or load_library(), name), args, keep)


def _i(v):
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{v} does not fit the 32 bits of the library's integer arguments")
    return ctypes.c_int32(v)


def prepare_route(cfg: RouteCfg, numTokens: int, logits, bias, expertIds, weights) -> PreparedCall:
    T, E, K = max(int(numTokens), 0), cfg.numExperts, cfg.numExpertPerToken
    args = [ctypes.byref(_b._cfg_copy(cfg)), _i(numTokens),
            _array(logits, T * E * _BYTES.get(cfg.dtype, 0), "logits", _FLOATS.get(cfg.dtype)),
            _array(bias, E * 4, "bias", "torch.float32"),
            _array(expertIds, T * K * 4, "expertIds", "torch.int32"),
            _array(weights, T * K * 4, "weights", "torch.float32")]
    return _call("epdc_route", args, (logits, bias, expertIds, weights))


def prepare_route_grad(cfg: RouteCfg, numTokens: int, logits, expertIds, dWeights, dLogits) -> PreparedCall:
    T, E, K = max(int(numTokens), 0), cfg.numExperts, cfg.numExpertPerToken
    row, kind = T * E * _BYTES.get(cfg.dtype, 0), _FLOATS.get(cfg.dtype)
    args = [ctypes.byref(_b._cfg_copy(cfg)), _i(numTokens), _array(logits, row, "logits", kind),
            _array(expertIds, T * K * 4, "expertIds", "torch.int32"),
            _array(dWeights, T * K * 4, "dWeights", "torch.float32"), _array(dLogits, row, "dLogits", kind)]
    return _call("epdc_route_grad", args, (logits, expertIds, dWeights, dLogits))


def epdc_mx_scale_dim(cols: int) -> int:
    return load_library().epdc_mx_scale_dim(min(max(int(cols), -1), 2 ** 31 - 1))


def _mx_sizes(numWindows, rowsPerWindow, cols):
    rows = max(int(numWindows), 0) * max(int(rowsPerWindow), 0)
    words = max(epdc_mx_scale_dim(cols), 0)
    return rows * int(cols), rows * (int(cols) // 2), rows * words * 4


def prepare_mx_quantize(numWindows: int, rowsPerWindow: int, cols: int, dtype: int, x, rowCount, q,
                        scales) -> PreparedCall:
    n, qb, sb = _mx_sizes(numWindows, rowsPerWindow, cols)
    args = [_i(numWindows), _i(rowsPerWindow), _i(cols), _i(dtype),
            _array(x, n * _BYTES.get(dtype, 0), "x", _FLOATS.get(dtype)),
            _array(rowCount, max(numWindows, 0) * 4, "rowCount", "torch.int32"), _array(q, qb, "q", size=1),
            _array(scales, sb, "scales", size=4)]
    return _call("epdc_mx_quantize", args, (x, rowCount, q, scales))


def prepare_mx_dequantize(numWindows: int, rowsPerWindow: int, cols: int, q, scales, rowCount, out,
                          outDtype: int) -> PreparedCall:
    n, qb, sb = _mx_sizes(numWindows, rowsPerWindow, cols)
    args = [_i(numWindows), _i(rowsPerWindow), _i(cols), _array(q, qb, "q", size=1),
            _array(scales, sb, "scales", size=4),
            _array(rowCount, max(numWindows, 0) * 4, "rowCount", "torch.int32"),
            _array(out, n * _BYTES.get(outDtype, 0), "out", _FLOATS.get(outDtype)), _i(outDtype)]
    return _call("epdc_mx_dequantize", args, (q, scales, rowCount, out))


def epdc_group_scratch_bytes(cfg: EpCfg, rank: int) -> int:
    return load_library().epdc_group_scratch_bytes(ctypes.byref(cfg), _i(rank))


def prepare_group_experts(cfg: EpCfg, rank: int, expertIds, weights, recvCount, offsets, entryRow, entryWeight, entryOf,
                          scratch, scratchBytes: int | None = None) -> PreparedCall:
    if scratchBytes is None:
        scratchBytes = 0 if scratch is None or isinstance(scratch, int) else scratch.numel() * scratch.element_size()
    W, M, K = (max(v, 0) for v in (cfg.worldSize, cfg.maxTokPerRank, cfg.numExpertPerToken))
    groups = (W if rank < 0 else 1) * max(cfg.numExpertPerRank, 0)
    n = W * M * K * 4
    w = n if cfg.useWeights else 0
    args = [ctypes.byref(_b._cfg_copy(cfg)), _i(rank), _array(expertIds, n, "expertIds", "torch.int32"),
            _array(weights, w, "weights", "torch.float32"), _array(recvCount, W * 4, "recvCount", "torch.int32"),
            _array(offsets, (groups + 1) * 4, "offsets", "torch.int32"),
            _array(entryRow, n, "entryRow", "torch.int32"), _array(entryWeight, w, "entryWeight", "torch.float32"),
            _array(entryOf, n, "entryOf", "torch.int32"), _array(scratch, int(scratchBytes), "scratch"),
            ctypes.c_size_t(int(scratchBytes))]
    return _call("epdc_group_experts", args,
                 (expertIds, weights, recvCount, offsets, entryRow, entryWeight, entryOf, scratch))


def prepare_expert_product(numExperts: int, numCols: int, hiddenDim: int, maxEntries: int, numRows: int, rows, rowScales,
                           offsets, entryRow, entryWeight, weights, weightScales, out, outDtype: int) -> PreparedCall:
    E, N, R, n = (max(int(v), 0) for v in (numExperts, numCols, numRows, maxEntries))
    rb, sb = max(int(hiddenDim), 0) // 2, max(epdc_mx_scale_dim(hiddenDim), 0) * 4
    args = [_i(numExperts), _i(numCols), _i(hiddenDim), _i(maxEntries), _i(numRows),
            _array(rows, R * rb, "rows", size=1), _array(rowScales, R * sb, "rowScales", size=4),
            _array(offsets, (E + 1) * 4, "offsets", "torch.int32"),
            _array(entryRow, n * 4, "entryRow", "torch.int32"),
            _array(entryWeight, n * 4, "entryWeight", "torch.float32"),
            _array(weights, E * N * rb, "weights", size=1), _array(weightScales, E * N * sb, "weightScales", size=4),
            _array(out, n * N * _BYTES.get(outDtype, 0), "out", _FLOATS.get(outDtype)), _i(outDtype)]
    return _call("epdc_expert_product", args,
                 (rows, rowScales, offsets, entryRow, entryWeight, weights, weightScales, out))


def epdc_route(cfg: RouteCfg, numTokens: int, logits, bias, expertIds, weights, stream=None, check: bool = True) -> int:
    return prepare_route(cfg, numTokens, logits, bias, expertIds, weights)(stream, check)


def epdc_route_grad(cfg: RouteCfg, numTokens: int, logits, expertIds, dWeights, dLogits, stream=None,
                    check: bool = True) -> int:
    return prepare_route_grad(cfg, numTokens, logits, expertIds, dWeights, dLogits)(stream, check)


def epdc_mx_quantize(numWindows: int, rowsPerWindow: int, cols: int, dtype: int, x, rowCount, q, scales, stream=None,
                     check: bool = True) -> int:
    return prepare_mx_quantize(numWindows, rowsPerWindow, cols, dtype, x, rowCount, q, scales)(stream, check)


def epdc_mx_dequantize(numWindows: int, rowsPerWindow: int, cols: int, q, scales, rowCount, out, outDtype: int,
                       stream=None, check: bool = True) -> int:
    return prepare_mx_dequantize(numWindows, rowsPerWindow, cols, q, scales, rowCount, out, outDtype)(stream, check)


def epdc_group_experts(cfg: EpCfg, rank: int, expertIds, weights, recvCount, offsets, entryRow, entryWeight, entryOf,
                       scratch, scratchBytes: int | None = None, stream=None, check: bool = True) -> int:
    return prepare_group_experts(cfg, rank, expertIds, weights, recvCount, offsets, entryRow, entryWeight, entryOf,
                                 scratch, scratchBytes)(stream, check)


def epdc_expert_product(numExperts: int, numCols: int, hiddenDim: int, maxEntries: int, numRows: int, rows, rowScales,
                        offsets, entryRow, entryWeight, weights, weightScales, out, outDtype: int, stream=None,
                        check: bool = True) -> int:
    return prepare_expert_product(numExperts, numCols, hiddenDim, maxEntries, numRows, rows, rowScales, offsets, entryRow,
                                  entryWeight, weights, weightScales, out, outDtype)(stream, check)
