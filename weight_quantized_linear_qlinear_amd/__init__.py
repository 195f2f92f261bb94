"""qlq: an MI355X (gfx950) quantized linear layer -- W8A16, W8A8-static and W8A8-dynamic GEMMs --
and the 8-bit operators between the linears of a decoder layer (norm to codes, norms of query and key
heads, rotary positions, the KV cache in 8 or 4 bits and attention over it).

The compute lives in libqlq.so (hand-written HIP kernels behind a C ABI,
include/qlq.h); this package is its Python binding.
"""
from .binding import (QTYPES, GRANULARITIES, QlqError, QuantizedKV, QuantizedKV4, QuantizedWeight,
                      calibrate_input_scale, code_dtype, gemm_plan, kv_append, kv_attention, kv_attention_workspace_bytes, kv_cache,
                      kv_dequantize, kv_gather, kv_quantize, lib, library_path, linear, linear_workspace_bytes, norm_rope, norm_rope_kv_append, packed_weight_bytes,
                      qlinear_w8a16, qlinear_w8a16_noalloc, qlinear_w8a8_dynamic, qlinear_w8a8_static, qlinear_w8a8_static_fused,
                      qlinear_w8a8_static_requant,
                      quantize_act_dynamic, quantize_act_static, quantize_weight, rms_norm,
                      rms_norm_quant_dynamic, rms_norm_quant_static, rope, rope_axes, rope_inv_freq, rope_kv_append,
                      scale_is_calibrated, unpack_weight, workspace_bytes)
from .graphs import DEFAULT_BUCKETS, GraphBuckets

__all__ = [
    "DEFAULT_BUCKETS", "GraphBuckets", "QTYPES", "GRANULARITIES", "QlqError", "QuantizedKV", "QuantizedKV4", "QuantizedWeight", "calibrate_input_scale", "code_dtype",
    "gemm_plan", "kv_append", "kv_attention", "kv_attention_workspace_bytes", "kv_cache", "kv_dequantize",
    "kv_gather", "kv_quantize", "linear", "linear_workspace_bytes",
    "lib", "library_path", "norm_rope", "norm_rope_kv_append", "packed_weight_bytes", "qlinear_w8a16", "qlinear_w8a16_noalloc", "qlinear_w8a8_dynamic",
    "qlinear_w8a8_static", "qlinear_w8a8_static_fused", "qlinear_w8a8_static_requant", "quantize_act_dynamic",
    "quantize_act_static",
    "quantize_weight", "rms_norm", "rms_norm_quant_dynamic", "rms_norm_quant_static", "rope", "rope_axes", "rope_inv_freq",
    "rope_kv_append", "scale_is_calibrated", "unpack_weight", "workspace_bytes",
]
