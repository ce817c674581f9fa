"""GB300-native (sm_103a) KDA recurrence: chunked prefill, in-place decode and
replay of accepted speculative-decode tokens; latent attention (expanded and
absorbed forms) and the paged cache it reads; the norm, the rotation, the attention
weight and the eviction of its rows.

The compute lives in ``libkda.so`` (hand-written CUDA kernels behind a C ABI,
``include/kda.h``); ``kda``, ``latent`` and ``rows`` are its thin Python bindings.
"""
from .kda import (KDAError, kda_chunk_fwd, kda_chunk_fwd_host, kda_chunk_fwd_noalloc,
                  kda_chunk_fwd_transitions,
                  kda_chunk_fwd_workspace_size, kda_decode_replay, kda_decode_step,
                  kda_post_fwd, kda_prep_fwd, kda_read_chunk_stats, kda_read_device_status,
                  kda_state_combine, kda_version, library, library_path)
from .latent import (kda_cache_copy_pages, kda_cache_write, kda_latent_bwd,
                     kda_latent_bwd_workspace_size, kda_latent_decode,
                     kda_latent_decode_workspace_size, kda_latent_fwd,
                     kda_latent_fwd_workspace_size)
from .rows import (kda_cache_evict, kda_cache_evict_workspace_size, kda_latent_weights,
                   kda_latent_weights_workspace_size, kda_norm_bwd, kda_norm_bwd_workspace_size,
                   kda_norm_fwd, kda_rope, kda_rope_inv_freq)

__all__ = ["KDAError", "kda_chunk_fwd", "kda_chunk_fwd_host", "kda_chunk_fwd_noalloc", "kda_chunk_fwd_transitions",
           "kda_chunk_fwd_workspace_size", "kda_decode_replay", "kda_decode_step",
           "kda_post_fwd", "kda_prep_fwd", "kda_read_chunk_stats", "kda_read_device_status",
           "kda_state_combine", "kda_version", "library", "library_path",
           "kda_cache_copy_pages", "kda_cache_write", "kda_latent_bwd",
           "kda_latent_bwd_workspace_size", "kda_latent_decode",
           "kda_latent_decode_workspace_size", "kda_latent_fwd",
           "kda_latent_fwd_workspace_size",
           "kda_cache_evict", "kda_cache_evict_workspace_size", "kda_latent_weights",
           "kda_latent_weights_workspace_size", "kda_norm_bwd", "kda_norm_bwd_workspace_size",
           "kda_norm_fwd", "kda_rope", "kda_rope_inv_freq"]
