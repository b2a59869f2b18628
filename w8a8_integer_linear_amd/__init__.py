"""INT8 W8A8 linear layer for quantized training on AMD MI355X (gfx950).

The compute path lives in libqlin.so (hand-written HIP kernels behind the C ABI
of include/qlin.h); this package only binds it for torch tensors.
"""
from ._native import (  # noqa: F401
    ACTIVATIONS, AdamWPlan, CK_BLOCK, lib, MAX_ADAPTERS, MAX_CONTRACTION, MAX_RANK,
    MFMA_CEILING_FRAG_BYTES, NOALLOC_SCRATCH_BYTES, QLIN_BF16, QLIN_F32, QLIN_OP_DW, QLIN_OP_DX,
    QLIN_OP_FWD, QlinError, SIGNATURES, qlin_act_bwd, qlin_act_bwd_ws_bytes, qlin_adamw_requant,
    qlin_adamw_tensors, qlin_adamw_tensors_plan, qlin_adapter_bwd, qlin_adapter_bwd_ws_bytes,
    qlin_adapter_fwd, qlin_adapter_fwd_ws_bytes, qlin_adapter_group, qlin_bwd_dw, qlin_bwd_dx,
    qlin_dequantize_weight, qlin_fwd, qlin_fwd_act, qlin_fwd_act_ws_bytes, qlin_fwd_gated,
    qlin_fwd_gated_ws_bytes, qlin_gemm_s32, qlin_hadamard, qlin_mfma_ceiling,
    qlin_product_noalloc, qlin_product_ws, qlin_product_ws_bytes, qlin_quantize_cols,
    qlin_quantize_grad, qlin_quantize_grad_scaled, qlin_quantize_rows, qlin_rmsnorm_bwd,
    qlin_rmsnorm_bwd_ws_bytes, qlin_rmsnorm_quant, qlin_sgd_requant, qlin_stream_copy,
    qlin_wn_init, qlin_wn_sgd_requant)
from .adapters import AdaptedLinearW8A8, pack_adapters  # noqa: F401
from .layer import LinearW8A8Training  # noqa: F401
from .mlp import MLPW8A8Training  # noqa: F401
