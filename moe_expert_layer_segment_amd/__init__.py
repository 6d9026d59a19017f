"""MI355X (gfx950) MoE expert layer with per-request LoRA deltas.

The compute runs in hand-written HIP kernels behind a C ABI
(``include/moe_lora.h``); :mod:`.binding` is a thin ctypes layer over it and
:mod:`.workloads` generates seeded synthetic inputs.
"""
from .binding import (  # noqa: F401
    compute_moe_lora_info,
    int8_block_m,
    moe_lora_align,
    moe_lora_align_capacity_rows,
    moe_lora_align_workspace_bytes,
    moe_lora_balance_loss,
    moe_lora_balance_loss_backward,
    moe_lora_balance_loss_workspace_bytes,
    moe_lora_dense_forward,
    moe_lora_dense_workspace_bytes,
    moe_lora_forward,
    moe_lora_forward_workspace_bytes,
    moe_lora_info,
    moe_lora_int8_dequantize,
    moe_lora_int8_gemm,
    moe_lora_int8_quantize,
    moe_lora_mx4_dequantize,
    moe_lora_mx4_gemm,
    moe_lora_mx4_quantize,
    moe_lora_permute,
    moe_lora_permute_backward,
    moe_lora_rms_norm_quantize,
    moe_lora_route,
    moe_lora_unpermute,
    moe_lora_unpermute_backward,
    mx4_block_m,
    run_dense,
    run_int8_layer,
    run_layer,
    run_mx4_layer,
)
