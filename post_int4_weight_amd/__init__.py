"""GPTQ / AWQ layer quantization on MI355X (gfx950): Python binding of libptq.so.

The compute path is the HIP library behind the C ABI in include/ptq.h; this
package only marshals torch tensors (device memory) and the current stream
into those calls. Importing it loads the library and fails loudly if it has
not been built (``python post_int4_weight_amd/build.py``).
"""
from .api import (PTQError, PTQ_BF16, PTQ_F32, library_path, hessian_workspace_bytes, hessian_accumulate,
                  gptq_factor_workspace_bytes, gptq_inverse_factor, gptq_columns_workspace_bytes,
                  gptq_quantize_columns, gptq_workspace_bytes, gptq_quantize_layer, awq_workspace_bytes,
                  awq_search_alpha, awq_gptq_quantize_layer, gptq_quantize_layer_zp, pack_int4,
                  dequantize_int4, layer_output_error_workspace_bytes, layer_output_error, quantize_tokens_int8,
                  matmul_int8_workspace_bytes, matmul_int8, linear_int8_workspace_bytes, linear_int8, KVCacheInt8,
                  kv_cache_write_int8, kv_cache_read_int8, attention_int8_cache_workspace_bytes,
                  attention_int8_cache, Rotary, rotary_apply, kv_cache_append_int8,
                  attention_int8_tree_workspace_bytes, attention_int8_tree, verify_drafts_workspace_bytes, verify_drafts)

__all__ = [
    "PTQError", "PTQ_BF16", "PTQ_F32", "library_path", "hessian_workspace_bytes", "hessian_accumulate",
    "gptq_factor_workspace_bytes", "gptq_inverse_factor", "gptq_columns_workspace_bytes",
    "gptq_quantize_columns", "gptq_workspace_bytes", "gptq_quantize_layer", "awq_workspace_bytes",
    "awq_search_alpha", "awq_gptq_quantize_layer", "gptq_quantize_layer_zp", "pack_int4", "dequantize_int4",
    "layer_output_error_workspace_bytes", "layer_output_error", "quantize_tokens_int8",
    "matmul_int8_workspace_bytes", "matmul_int8", "linear_int8_workspace_bytes", "linear_int8", "KVCacheInt8",
    "kv_cache_write_int8", "kv_cache_read_int8", "attention_int8_cache_workspace_bytes", "attention_int8_cache",
    "Rotary", "rotary_apply", "kv_cache_append_int8", "attention_int8_tree_workspace_bytes", "attention_int8_tree",
    "verify_drafts_workspace_bytes", "verify_drafts",
]
