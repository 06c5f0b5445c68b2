"""Gated delta-rule recurrence (Gated DeltaNet / Gated DeltaNet-2) and the softmax-attention layer of its
hybrid stacks for B200 (sm_100a).

The compute path is libgdn.so (CUDA kernels behind the C ABI in include/gdn.h); this package
only marshals arguments.  See gdn.py for the calls.
"""
from .gdn import (GdnError, gdn_attn_bwd, gdn_attn_decode, gdn_attn_fwd, gdn_attn_fwd_cache_size, gdn_chunk_bwd,
                  gdn_chunk_fwd, gdn_chunk_fwd_noalloc, gdn_decode_step, gdn_kv_append, gdn_layer_core_fwd,
                  gdn_qk_norm_rope_bwd, gdn_qk_norm_rope_fwd, load)

__all__ = ["GdnError", "gdn_chunk_fwd", "gdn_chunk_fwd_noalloc", "gdn_chunk_bwd", "gdn_decode_step", "gdn_layer_core_fwd",
           "gdn_qk_norm_rope_fwd", "gdn_qk_norm_rope_bwd", "gdn_attn_fwd_cache_size", "gdn_attn_fwd", "gdn_attn_bwd",
           "gdn_kv_append", "gdn_attn_decode", "load"]
