"""mxfp4_block_fake_b200: MXFP4 block fake quantisation (QDQ + clipped STE) on
NVIDIA B200, behind the C ABI of include/mxfp4.h (libmxfp4.so).

Layers:
  libmxfp4.so         sm_100a kernels + C ABI (csrc/mxfp4.cu)
  _abi                ctypes mirror of the C ABI
  ops                 the entry points over torch CUDA tensors
  qat                 autograd STE function, quantizer module, QAT Linear
  moe                 differentiable routing, dispatch, combine and grouped linear; MoE module
  workloads           seeded synthetic inputs
"""
from ._abi import MXFP4ArgumentError, MXFP4Error
from .moe import MXFP4MoE, moe_combine, moe_dispatch, moe_expert_operands, moe_grouped_linear, moe_route
from .ops import (
    DispatchResult,
    DualLevelResult,
    LinearResult,
    QDQResult,
    RouteResult,
    colwise_scale_rows_bound,
    mxfp4_colwise_scale_rows,
    mxfp4_dual_level_qdq,
    mxfp4_grouped_gemm,
    mxfp4_grouped_linear,
    mxfp4_grouped_linear_bwd,
    mxfp4_moe_combine,
    mxfp4_moe_combine_bwd,
    mxfp4_moe_dispatch,
    mxfp4_moe_route,
    mxfp4_moe_route_bwd,
    mxfp4_qdq_fwd,
    mxfp4_qdq_fwd_bwd,
    mxfp4_ste_bwd,
)
from .qat import (
    MXFP4FakeQuantizer,
    MXFP4QATConfig,
    MXFP4QATLinear,
    convert_to_mxfp4_qat,
    mxfp4_fake_quant,
    mxfp4_quant_dequant,
    mxfp4_saturation_mask,
    unpack_mask,
)

__all__ = [
    "MXFP4Error", "MXFP4ArgumentError", "QDQResult", "DualLevelResult", "mxfp4_dual_level_qdq", "colwise_scale_rows_bound", "mxfp4_colwise_scale_rows",
    "mxfp4_qdq_fwd", "mxfp4_qdq_fwd_bwd", "mxfp4_ste_bwd", "MXFP4FakeQuantizer", "MXFP4QATConfig",
    "MXFP4QATLinear", "convert_to_mxfp4_qat", "mxfp4_fake_quant", "mxfp4_quant_dequant",
    "mxfp4_saturation_mask", "unpack_mask", "DispatchResult", "LinearResult", "RouteResult", "mxfp4_grouped_gemm",
    "mxfp4_grouped_linear", "mxfp4_grouped_linear_bwd", "mxfp4_moe_combine", "mxfp4_moe_combine_bwd",
    "mxfp4_moe_dispatch", "mxfp4_moe_route", "mxfp4_moe_route_bwd", "MXFP4MoE", "moe_combine", "moe_dispatch",
    "moe_expert_operands", "moe_grouped_linear", "moe_route",
]
