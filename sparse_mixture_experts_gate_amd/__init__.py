"""DeepSeekMoE feed-forward layer on one MI355X (gfx950): HIP kernels behind a
C ABI (include/dsmoe.h, include/dsmoe_ops.h for the operators around the layer
and include/dsmoe_tokens.h for those on a token's way through it), with this
thin Python binding on top."""
from ._lib import (MOE_DT_BF16, MOE_DT_F32, MOE_DT_FP8_E4M3, MoeError, MoeLayerDesc, MoeWeights,
                   deepseek_moe_forward, deepseek_moe_forward_noalloc, lib, make_weights, moe_abi_version, moe_bias_update,
                   moe_combine, moe_expert_ffn, moe_gate, moe_permute, moe_profile_events, moe_quantize_fp8_blocks,
                   moe_quantize_fp8_rows, moe_route_from_logits, moe_workspace_size,
                   moe_backward, moe_backward_workspace_size, moe_forward_train,
                   moe_seq_balance_loss, moe_seq_balance_workspace_size,
                   moe_backward_fp8, moe_transpose_fp8_blocks)
from ._ops import (MOE_GROUPED_DGRAD, MOE_GROUPED_FORWARD, MOE_GROUPED_WGRAD, MoeGroupedDesc,
                   MoeNormDesc, MoeOrthDesc, moe_grouped_gemm, moe_grouped_gemm_dgrad,
                   moe_grouped_gemm_wgrad, moe_grouped_gemm_workspace_size, moe_layernorm_backward,
                   moe_layernorm_backward_workspace_size, moe_layernorm_forward,
                   moe_orthogonalize, moe_orthogonalize_workspace_size)
from ._token_ops import (MOE_MX4_PLAIN, MOE_MX4_SWIGLU, MoeDispatchDesc, MoeMx4Desc, MoeMx4GemmDesc,
                         MoeRmsNormDesc, moe_mx4_dequantize, moe_mx4_gemm, moe_mx4_quantize,
                         moe_rmsnorm_backward, moe_rmsnorm_backward_workspace_size,
                         moe_rmsnorm_forward, moe_token_combine, moe_token_combine_backward,
                         moe_token_dispatch, moe_token_dispatch_workspace_size)
from .blocks import GroupedLinear, LayerNorm, Muon
from .layer import MoELayer, make_desc, quantize_fp8_blocks
from .tokens import MX4Linear, RMSNorm, TokenDispatch, mx4_dequantize, mx4_quantize
from .workloads import CONFIGS, Workload, make_inputs, make_layer, make_tokens

__all__ = [
    "MOE_DT_BF16", "MOE_DT_F32", "MOE_DT_FP8_E4M3", "MoeError", "MoeLayerDesc", "MoeWeights",
    "deepseek_moe_forward", "deepseek_moe_forward_noalloc", "lib", "make_weights", "moe_abi_version", "moe_bias_update",
    "moe_combine", "moe_expert_ffn", "moe_gate", "moe_permute", "moe_profile_events", "moe_quantize_fp8_blocks",
    "moe_quantize_fp8_rows", "moe_route_from_logits", "moe_workspace_size", "MoELayer",
    "make_desc", "quantize_fp8_blocks", "CONFIGS", "Workload", "make_inputs", "make_layer",
    "make_tokens", "moe_backward", "moe_backward_workspace_size", "moe_forward_train",
    "moe_seq_balance_loss", "moe_seq_balance_workspace_size", "moe_backward_fp8",
    "moe_transpose_fp8_blocks",
    "MOE_GROUPED_DGRAD", "MOE_GROUPED_FORWARD", "MOE_GROUPED_WGRAD",
    "moe_grouped_gemm_workspace_size", "MoeGroupedDesc", "MoeNormDesc", "MoeOrthDesc", "moe_grouped_gemm", "moe_grouped_gemm_dgrad",
    "moe_grouped_gemm_wgrad", "moe_layernorm_backward", "moe_layernorm_backward_workspace_size",
    "moe_layernorm_forward", "moe_orthogonalize", "moe_orthogonalize_workspace_size",
    "GroupedLinear", "LayerNorm", "Muon",
    "MOE_MX4_PLAIN", "MOE_MX4_SWIGLU", "MoeDispatchDesc", "MoeMx4Desc", "MoeMx4GemmDesc",
    "MoeRmsNormDesc", "moe_mx4_dequantize", "moe_mx4_gemm", "moe_mx4_quantize",
    "moe_rmsnorm_backward", "moe_rmsnorm_backward_workspace_size", "moe_rmsnorm_forward",
    "moe_token_combine", "moe_token_combine_backward", "moe_token_dispatch",
    "moe_token_dispatch_workspace_size", "MX4Linear", "RMSNorm", "TokenDispatch",
    "mx4_dequantize", "mx4_quantize",
]
