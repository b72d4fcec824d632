"""B200-native (sm_100a) Sparse-BitNet BitLinear path.

The functions below are thin bindings of the C ABI in include/bitlinear.h; the
library libbitlinear.so is loaded on first use and its absence is an error.
"""
from .bitlinear import (  # noqa: F401
    BL_GRADW_DEQUANT_X,
    BL_OUT_BF16,
    BL_OUT_F32,
    bitlinear_abi_version,
    bitlinear_act_quant,
    bitlinear_bwd,
    bitlinear_bwd_workspace_size,
    bitlinear_device_status,
    bitlinear_fwd,
    bitlinear_fwd_grouped,
    bitlinear_grad_x_i8,
    bitlinear_grad_x_i8_workspace_size,
    bitlinear_mask_threshold_hist,
    bitlinear_quant_mask,
    bitlinear_quant_mask_noalloc,
    bitlinear_quant_mask_status,
    bitlinear_quant_mask_workspace_size,
    bitlinear_sgd_quant_mask,
    bitlinear_grad_w_grouped,
    sp_meta_shape,
)
from .head import (  # noqa: F401
    BL_FP8_E4M3,
    BL_FP8_E5M2,
    bitlinear_fp8_bwd,
    bitlinear_fp8_fwd,
    bitlinear_fp8_fwd_workspace_size,
    bitlinear_fp8_quant,
    bitlinear_fp8_quant_weight,
    bitlinear_linear_ce_bwd,
    bitlinear_linear_ce_bwd_workspace_size,
    bitlinear_linear_ce_fwd,
    bitlinear_linear_ce_fwd_workspace_size,
    fp8_scales_shape,
)
