"""GB300-native fused inverse RoPE + VHA postmix (forward / backward) and the
sparse-attention KV index remap, and the paged latent cache with the attention
that reads it, as hand-written sm_103a CUDA kernels behind a C ABI
(``include/invrope.h``, ``include/latent_attn.h``), with a thin ctypes binding
of the same names.
"""

from .binding import (  # noqa: F401
    KV_LATENT_BF16,
    KV_LATENT_E4M3,
    InvropeError,
    invrope_debug_occupy_next_slot,
    invrope_postmix_bwd,
    invrope_postmix_bwd_ex,
    invrope_postmix_bwd_noalloc,
    invrope_postmix_bwd_workspace_bytes,
    invrope_postmix_fwd,
    invrope_postmix_fwd_ex,
    invrope_take_device_fault,
    invrope_watchdog_selftest,
    kv_idx_local_to_global,
    kv_idx_local_to_global_i64,
    kv_latent_empty,
    kv_latent_read,
    kv_latent_row_bytes,
    kv_latent_write,
    latent_attn_decode,
    latent_attn_sparse,
    latent_attn_workspace_bytes,
    lib,
    lib_path,
)
