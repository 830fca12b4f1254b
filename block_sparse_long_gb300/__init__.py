"""CoSA block-sparse long-context prefill for GB300 (sm_103a).

The hot path lives in libcosa.so (CUDA kernels behind the C ABI of include/cosa.h);
``block_sparse_long_gb300.cosa`` is its thin Python binding.  What stands around it - query/key norms with
rotation and the cache write, the 4-bit cache, decode attention over it, eviction - lives in libcosa_kv.so
(include/cosa_kv.h) and ``block_sparse_long_gb300.kv``.
"""
from .cosa import (COSA_OK, COSA_ERR_INVALID_ARG, COSA_ERR_UNSUPPORTED, COSA_ERR_CUDA, COSA_ERR_DEVICE_TIMEOUT,
                   COSA_ERR_WORKSPACE, COSA_ERR_BAD_INPUT, VISIT_COMPUTED, VISIT_SKIPPED, VISIT_IGNORED, EXPORTS,
                   CosaError, CosaParams, cosa_prefill_workspace_size, cosa_proxy_select, cosa_proxy_select_static,
                   cosa_proxy_workspace_size, cosa_sparse_prefill, cosa_status_string, cosa_version, library,
                   make_params, params_for, stage1_pitch)
from .kv import (COSA_KV_FLAG_INTERLEAVED, KV_EXPORTS, CosaKvParams, cosa_kv4_attention,
                 cosa_kv4_attention_workspace_size, cosa_kv4_evict, cosa_kv4_load, cosa_kv4_store, cosa_kv_version,
                 cosa_qk_norm_rope, kv4_cache_shape, kv_library, make_kv_params)

__all__ = [n for n in dir() if n.startswith(("cosa_", "COSA_", "VISIT_")) or n in (
    "CosaError", "CosaParams", "EXPORTS", "library", "make_params", "params_for", "stage1_pitch", "CosaKvParams",
    "KV_EXPORTS", "kv_library", "kv4_cache_shape", "make_kv_params")]
