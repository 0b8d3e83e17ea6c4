"""W4A4 group-quantized GEMM, MXFP4 GEMM, NVFP4 GEMM, W8A8 GEMM with what an 8-bit
feed-forward block needs around it, and attention over an INT8 key/value cache for
MI355X (gfx950).

The compute lives in ``libw4a4.so`` (hand-written HIP kernels behind a C ABI, declared
in ``include/w4a4.h``, ``include/ffn8.h`` and ``include/kv8.h``). The Python side only marshals arguments; the
tensor-level entry points (same names as the C ABI) are in :mod:`.ops` and are
re-exported here on first use.
"""
_OPS = (
    "w4a4_quantize_act", "w4a4_pack_weight", "w4a4_gemm", "w4a4_gemm_splitk", "w4a4_gemm_debug_partials",
    "mxfp4_quantize", "mxfp4_quantize_residual", "mxfp4_quantize_append_copy",
    "mxfp4_gemm", "mxfp4_gemm_debug_partials",
    "nvfp4_global_scale", "nvfp4_quantize", "nvfp4_gemm", "nvfp4_gemm_debug_partials",
    "w8a8_quantize_act", "w8a8_pack_weight", "w8a8_gemm", "w8a8_linear",
    "w8a8_rmsnorm_quantize", "w8a8_gemm_act", "w8a8_linear_act", "w8a8_pack_gated", "moe_route", "w8a8_moe",
    "kv8_new_cache", "kv8_append", "kv8_gather", "kv8_attention",
)


def __getattr__(name):
    if name in _OPS:
        from . import ops
        return getattr(ops, name)
    raise AttributeError(name)
