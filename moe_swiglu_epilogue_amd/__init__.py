"""MI355X (gfx950) fused SwiGLU + NVFP4 block quantization.

The compute lives in ``libmoe_nvfp4.so`` (hand-written HIP kernels behind a
C ABI, declared in ``include/moe_nvfp4.h``); this package is a thin binding:
``nvfp4_quantize``, ``swiglu_nvfp4_quantize`` and ``nvfp4_dequantize`` take
torch tensors on the GPU, marshal pointers, sizes and the current stream, and
call the library. Importing the package does not load the library; the first
call does, and raises if it is missing. The operators of a decoding step
(``kv_block_tables``, ``nvfp4_paged_attention``, ``moe_layer_nvfp4``,
``moe_layer_bf16``; ``include/nvfp4_serving.h``) and those of sparse attention
over the cache (``nvfp4_rope_append``, ``nvfp4_page_keys``,
``nvfp4_select_pages``, ``nvfp4_sparse_attention``; ``include/nvfp4_sparse.h``)
are in the same library.
"""
import importlib

__all__ = ["nvfp4_quantize", "swiglu_nvfp4_quantize", "nvfp4_dequantize",
           "nvfp4_global_scale", "swiglu_nvfp4_global_scale", "swiglu_bf16",
           "moe_l1_gemm_swiglu_nvfp4", "moe_l1_gemm_bf16", "nvfp4_quantize_paged",
           "nvfp4_dequantize_paged", "Nvfp4Error", "library_path",
           "kv_block_tables", "nvfp4_paged_attention", "moe_layer_nvfp4", "moe_layer_bf16",
           "nvfp4_rope_append", "nvfp4_page_keys", "nvfp4_select_pages", "nvfp4_sparse_attention"]
_SERVING = ("kv_block_tables", "nvfp4_paged_attention", "moe_layer_nvfp4", "moe_layer_bf16")
_SPARSE = ("nvfp4_rope_append", "nvfp4_page_keys", "nvfp4_select_pages", "nvfp4_sparse_attention")


def __getattr__(name):
    if name == "serving" or name in _SERVING:
        module = importlib.import_module(__name__ + ".serving")
    elif name == "sparse" or name in _SPARSE:
        module = importlib.import_module(__name__ + ".sparse")
    elif name == "binding" or name in __all__:
        module = importlib.import_module(__name__ + ".binding")
    else:
        raise AttributeError(name)
    value = module if name in ("binding", "serving", "sparse") else getattr(module, name)
    globals()[name] = value      # found at once from now on
    return value
