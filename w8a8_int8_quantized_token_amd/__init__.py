"""MI355X-native fused W8A8 linear (per-token int8 activations x
per-output-channel int8 weights -> int32 on the matrix cores -> dequant +
bias epilogue -> bf16), a thin torch binding over libw8a8.so.

The method is the one in the abstract of "Realizing Native INT8 Compute for
Diffusion Transformers on Consumer GPUs: A Fused INT8 GEMM Kernel for
Ideogram 4.0" (arXiv 2606.14598).
"""
from ._lib import LIB_PATH, MAX_K, W8A8Error, lib, status_str
from .block_ops import (gated_linear, gated_linear_backward, gated_linear_dynamic, linear_backward, linear_dynamic,
                        qk_norm_rope, qk_norm_rope_backward)
from .adapter_ops import (add_rms_norm_backward, add_rms_norm_quantize, linear_adapters, linear_adapters_backward,
                          linear_adapters_dynamic)
from .autograd import gated_linear_ste, linear_ste
from .module import Tokens, W8A8AdaptedLinear, W8A8GatedMLP, W8A8Linear, W8A8QKV, W8A8RMSNorm
from .ops import (dequantize_rows, gemm_f32_fp8, gemm_i32, linear, linear_fp8, linear_splitk,
                  mfma_ceiling, num_tiles, select_splitk, splitk_workspace_bytes,
                  quantize_act, quantize_act_fp8, quantize_weight, quantize_weight_fp8,
                  select_tile, tile_info)
from .slowpath import dequant_bf16_linear

__all__ = ["LIB_PATH", "MAX_K", "Tokens", "W8A8AdaptedLinear", "W8A8Error", "W8A8GatedMLP", "W8A8Linear", "W8A8QKV",
           "W8A8RMSNorm", "add_rms_norm_backward",
           "add_rms_norm_quantize", "dequant_bf16_linear",
           "dequantize_rows", "gated_linear", "gated_linear_backward", "gated_linear_dynamic", "gated_linear_ste",
           "gemm_f32_fp8", "gemm_i32",
           "lib", "linear", "linear_adapters", "linear_adapters_backward",
           "linear_adapters_dynamic", "linear_backward", "linear_dynamic",
           "linear_fp8", "linear_splitk", "linear_ste",
           "mfma_ceiling", "select_splitk", "splitk_workspace_bytes",
           "num_tiles", "qk_norm_rope", "qk_norm_rope_backward", "quantize_act", "quantize_act_fp8", "quantize_weight",
           "quantize_weight_fp8", "select_tile", "status_str", "tile_info"]
