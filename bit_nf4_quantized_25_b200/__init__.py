"""NF4 + double-quantisation + LoRA linear layer for B200 (sm_100a).

The computation lives in ``libqlora_nf4.so`` (C ABI: ``include/qlora_nf4.h``); the
``binding`` module marshals torch tensors into it. Importing the package does not load
the library; the first call does, and fails loudly if it is missing.
"""
from .binding import (Act8, Int4Weight, NF4Weight, QNError, act8_dequantize, act8_quantize, act8_sizes,
                      int4_dequantize, int4_linear_fwd, int4_quantize, int4_sizes, launch_count,
                      linear_workspace_size, load, lora_grads_act8_workspace_size, lora_grads_workspace_size,
                      new_workspace, nf4_dequantize, nf4_quantize, nf4_quantize_static_ws, qlora_linear_bwd_x,
                      qlora_linear_fwd, qlora_lora_grads, qlora_lora_grads_act8, qlora_merge_bf16,
                      quantize_workspace_size, sizes, swiglu_act8_bwd, swiglu_act8_fwd, weight_sizes, workspace_check)

__all__ = ["Act8", "Int4Weight", "NF4Weight", "QNError", "act8_dequantize", "act8_quantize", "act8_sizes",
           "int4_dequantize", "int4_linear_fwd", "int4_quantize", "int4_sizes", "launch_count",
           "linear_workspace_size", "load", "lora_grads_act8_workspace_size", "lora_grads_workspace_size",
           "new_workspace", "nf4_dequantize", "nf4_quantize", "nf4_quantize_static_ws", "qlora_linear_bwd_x",
           "qlora_linear_fwd", "qlora_lora_grads", "qlora_lora_grads_act8", "qlora_merge_bf16",
           "quantize_workspace_size", "sizes", "swiglu_act8_bwd", "swiglu_act8_fwd", "weight_sizes",
           "workspace_check"]
