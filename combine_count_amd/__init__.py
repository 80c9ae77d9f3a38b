"""MI355X-native MoE expert-parallel dispatch + combine (one GPU's share),
with the operators on both sides of them: routing, fp4x2 quantisation,
grouping by expert, the experts' product, and the experts in bf16 and int8
with their gradients.

The compute path is libepdc.so (hand-written HIP for gfx950) behind the C
ABI in include/epdc.h; this package is its Python binding.
"""
from .binding import (EPDC_BF16, EPDC_FP4X2, EPDC_FP8, EPDC_FP32, EPDC_MAX_EXPERT_DIM, EPDC_MAX_EXPERT_ENTRIES,
                      EPDC_MAX_GROUP_EXPERTS, EPDC_MAX_ROUTE_EXPERTS, EPDC_MAX_SCALE_DIM, EPDC_SIGMOID, EPDC_SOFTMAX,
                      EPDC_STATUS_ROW_OUTSIDE, EPDC_STATUS_WAIT_TIMEOUT, EPDC_STATUS_WORD, EXPORTS, EpCfg, EpdcError,
                      PreparedCall, RouteCfg, dispatch_status, epdc_combine, epdc_combine_push, epdc_combine_reduce,
                      epdc_dispatch, epdc_dispatch_noalloc, epdc_dispatch_scratch_bytes, epdc_landing_rows,
                      epdc_last_error, load_library, prepare_combine, prepare_combine_push, prepare_combine_reduce,
                      prepare_dispatch)
from .buffers import DispatchBuffers, LandingBuffers
from .expert_ops import (epdc_expert_gate, epdc_expert_gate_grad, epdc_expert_gate_int, epdc_expert_linear,
                         epdc_expert_linear_int, epdc_expert_rows_grad, epdc_expert_weights_grad, epdc_int_quantize,
                         prepare_expert_gate, prepare_expert_gate_grad, prepare_expert_gate_int,
                         prepare_expert_linear, prepare_expert_linear_int, prepare_expert_rows_grad,
                         prepare_expert_weights_grad, prepare_int_quantize)
from .layer_ops import (epdc_expert_product, epdc_group_experts, epdc_group_scratch_bytes, epdc_mx_dequantize,
                        epdc_mx_quantize, epdc_mx_scale_dim, epdc_route, epdc_route_grad, prepare_expert_product,
                        prepare_group_experts, prepare_mx_dequantize, prepare_mx_quantize, prepare_route,
                        prepare_route_grad)

__all__ = ["EPDC_BF16", "EPDC_FP32", "EPDC_FP8", "EPDC_FP4X2", "EPDC_MAX_SCALE_DIM", "EPDC_STATUS_WORD",
           "EPDC_STATUS_WAIT_TIMEOUT", "EPDC_STATUS_ROW_OUTSIDE", "EXPORTS", "EpCfg", "EpdcError",
           "dispatch_status", "epdc_combine", "epdc_combine_push", "epdc_dispatch_noalloc",
           "epdc_combine_reduce", "epdc_dispatch", "epdc_dispatch_scratch_bytes", "epdc_landing_rows",
           "epdc_last_error", "load_library", "DispatchBuffers", "LandingBuffers", "PreparedCall",
           "prepare_dispatch", "prepare_combine", "prepare_combine_push", "prepare_combine_reduce",
           "EPDC_SOFTMAX", "EPDC_SIGMOID", "EPDC_MAX_ROUTE_EXPERTS", "EPDC_MAX_GROUP_EXPERTS", "RouteCfg",
           "epdc_route", "epdc_route_grad", "epdc_mx_scale_dim", "epdc_mx_quantize", "epdc_mx_dequantize",
           "epdc_group_scratch_bytes", "epdc_group_experts", "epdc_expert_product", "prepare_route",
           "prepare_route_grad", "prepare_mx_quantize", "prepare_mx_dequantize", "prepare_group_experts",
           "prepare_expert_product", "EPDC_MAX_EXPERT_DIM", "EPDC_MAX_EXPERT_ENTRIES",
           "epdc_expert_linear", "epdc_expert_rows_grad",
           "epdc_expert_weights_grad", "epdc_expert_gate", "epdc_expert_gate_grad", "epdc_int_quantize",
           "epdc_expert_gate_int", "epdc_expert_linear_int", "prepare_expert_linear",
           "prepare_expert_rows_grad", "prepare_expert_weights_grad", "prepare_expert_gate",
           "prepare_expert_gate_grad", "prepare_int_quantize", "prepare_expert_gate_int",
           "prepare_expert_linear_int"]
