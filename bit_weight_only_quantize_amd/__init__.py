"""MI355X-native AWQ W4A16: group-quantized linear layer, alpha-grid scale search,
and attention over a key/value cache in the same 4-bit group format.

The compute lives in libawq355.so (HIP kernels for gfx950 behind a C ABI,
include/awq355.h); this package is its ctypes binding.  Build the library with
``python -m bit_weight_only_quantize_amd.build``.  Accessing any API name
loads the library and raises ImportError if it is not built.
"""

_API = (
    "awq_quantize_pack", "awq_dequantize", "awq_linear", "awq_linear_ex", "awq_linear_ws", "awq_linear_noalloc",
    "awq_linear_fused", "awq_linear_fused_workspace_size", "AWQ_EPILOGUE_NONE",
    "AWQ_EPILOGUE_SILU_MUL", "AWQ_MAX_PARTS",
    "awq_linear_epilogue", "ACTIVATIONS",
    "awq_linear_workspace_size", "awq_scale_search",
    "awq_scale_search_workspace_size", "AwqError", "config", "empty_packed", "lib",
    "AWQ_F16", "AWQ_BF16", "AWQ_F32", "AWQ_KERNEL_AUTO", "AWQ_KERNEL_GEMV",
    "AWQ_KERNEL_GEMM", "AWQ_KERNEL_BATCHED", "AWQ_GEMV_MAX_M", "AWQ_BATCHED_MAX_M", "EXPORTS",
    "LIB_PATH", "empty_kv_cache", "awq_kv_assign", "awq_kv_append", "awq_kv_gather",
    "awq_kv_attention", "awq_kv_attention_workspace_size",
    "awq_kv_copy_pages", "awq_kv_fork", "awq_kv_release", "awq_kv_release_workspace_size",
    "awq_kv_compact", "awq_kv_compact_workspace_size",
    "awq_rope_frequencies", "awq_rope", "awq_kv_append_rope", "ROPE_SCALINGS", "AWQ_ROPE_MAX_DIM",
)

__all__ = list(_API)


def __getattr__(name):
    if name in _API:
        from . import binding
        value = globals()[name] = getattr(binding, name)      # (later accesses find it at once)
        return value
    raise AttributeError(name)
