"""FP8-quantised paged decode attention for GB300 (sm_103a).

Two calls, both hand-written CUDA kernels behind a C ABI (``include/fp8pa.h``):

* ``kv_append_quant`` -- absmax-scale each new token's K/V rows, round them
  to E4M3 or E5M2 (or symmetric INT8 codes) and scatter codes and scales
  into the paged cache.
* ``paged_decode_attention`` -- grouped-query (or shared-latent MLA)
  attention of one query token per request over its paged FP8 cache, split
  across the GPU and merged.

Around them: ``kv_append_rope`` turns q and K by rotary positions on the way
into the cache, ``paged_decode_attention_mod`` decodes with a sliding window,
an always-visible prefix, capped scores or a distance bias, and
``paged_prefill_attention`` attends ragged query chunks of any length under
the same score modifiers, ``paged_tree_attention`` trees of drafted tokens.  ``kv_keep_accepted``, ``kv_fork``, ``kv_resize`` and
``kv_compact`` keep the pages of sequences that branch.

The torch-facing wrappers live in :mod:`.binding` and are re-exported here
on first use, so that importing the input generators (:mod:`.workloads`)
does not need the native library.  Using any wrapper loads ``libfp8pa.so``
and raises if it is missing: there is no fallback path.
"""
_API = ("kv_append_quant", "kv_append_quant_segment", "segment_scale_heads",
        "kv_channel_scales", "kv_channel_absmax_update",
        "kv_scales_from_absmax", "paged_decode_attention", "paged_multiquery_attention",
        "decode_step", "kv_append_rope", "paged_decode_attention_mod", "paged_prefill_attention",
        "prefill_workspace_bytes",
        "paged_tree_attention", "tree_workspace_bytes", "MAX_TREE",
        "KvPages", "kv_keep_accepted", "kv_fork", "kv_resize", "kv_compact",
        "pages_workspace_bytes",
        "decode_workspace_bytes", "get_device_error", "set_decode_workers", "version",
        "E4M3", "E5M2", "INT8", "SCALE_TOKEN_HEAD", "SCALE_CHANNEL_STATIC", "SCALE_TOKEN_GROUP",
        "SCALE_MX_BLOCK", "SCALE_SEGMENT", "SEGMENT_TOKENS",
        "OUT_BF16", "OUT_F32", "Fp8paError")

__all__ = list(_API)


def __getattr__(name):
    if name in _API:
        from . import binding
        value = globals()[name] = getattr(binding, name)  # found at once from now on
        return value
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
