"""Fused 4-bit AdamW optimizer step for MI355X (gfx950).

This package is a thin ctypes binding of the C ABI in ``include/q4adamw.h``
(``libq4adamw.so``): it marshals arguments and nothing else.  Every step of
the optimizer runs in the library's HIP kernels; PyTorch only provides device
memory and the current stream.  Importing works anywhere; loading the
library (first call) raises when it has not been built.
"""
from __future__ import annotations

from .api import (  # noqa: F401
    Q4Config, Q4HParams, Q4Tensor, Q4StateBytes, Q4StateHeader, Q4Error, load_library,
    q4adamw_abi_version, q4adamw_status_string, q4adamw_last_error, q4adamw_default_config,
    q4adamw_validate, q4adamw_workspace_bytes, q4adamw_state_bytes, q4adamw_make_header,
    q4adamw_check_header, q4adamw_host_scalars, q4adamw_codebook, q4adamw_init_state, q4adamw_step,
    q4adamw_dequant_state, q4adamw_flat_offsets, q4adamw_accumulate, q4adamw_grad_stats, q4adamw_grad_norm,
    RECIPE_ZIP_SR, RECIPE_ZE_EDEN, RECIPE_FACTORED, RECIPE_FP32, RECIPE_CUSTOM, RECIPE_BLOCK8,
    CB_NF4, CB_SDYN4, CB_DYN4, CB_DYN4_NZ, CB_LIN4_NZ, CB_SDYN8, CB_DYN8,
    RULE_STATE_RTN, RULE_STATE_SR, RULE_UPDATE_RTN, RULE_UPDATE_SR,
    HP_REUSE_TABLE, HP_CHECK_POINTERS, HP_GRAD_STATS, ACC_FIRST, ACC_LAST, ACC_REUSE_TABLE, TF_LM_HEAD,
)
from .api import (  # noqa: F401
    Q4MXMatrix, q4mx_matrix_bytes, q4mx_quantize, q4mx_dequantize, q4mx_linear, q4mx_linear_workspace_bytes,
    q4mx_linear_bf16, q4mx_linear_bf16_workspace_bytes, q4mx_dgrad, q4mx_dgrad_workspace_bytes, q4mx_wgrad,
    q4mx_wgrad_workspace_bytes, q4mx_act_forward, q4mx_act_backward, MX_FP4, MX_FP8, MX_F32, MX_BF16, MX_GELU,
    MX_GELU_ERF, MX_SWIGLU, MX_WGRAD_TRANSPOSED, MX_WGRAD_ADD, MX_FEW_TOKENS,
)
from .api import (  # noqa: F401
    Q4NNHeads, Q4NNRope, q4nn_embedding, q4nn_embedding_mx, q4nn_embedding_grad, q4nn_embedding_grad_workspace_bytes,
    q4nn_head_norm_rope, q4nn_head_norm_rope_backward, q4nn_head_norm_rope_backward_workspace_bytes, q4nn_dropout,
    NN_I32, NN_I64, NN_ADD,
)
from .state import Q4State, RECIPE_BY_NAME  # noqa: F401
from . import mx  # noqa: F401
from . import layers  # noqa: F401
