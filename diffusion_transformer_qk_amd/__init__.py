"""Fused diffusion-transformer QK-norm + RoPE (with the AdaLN modulation and the
VAE group norm + SiLU steps, attention, layer norm, and the backward passes of
all but the VAE step) for AMD Instinct MI355X (gfx950).

The passes run in hand-written HIP kernels behind the C ABI of
``include/qknorm_rope.h``, ``include/fuse_scale_shift.h``,
``include/group_norm_silu.h``, ``include/dit_attention.h``,
``include/layer_norm.h`` and ``include/qknorm_rope_backward.h``
(``libqknorm_rope.so`` and the ``libdit_attention.so`` it loads); this package is the thin Python binding over it.
"""
from .binding import (  # noqa: F401
    EXPORTS, LIB_PATH, QkrError, attention, attention_backward, attention_workspace_size,
    dit_fuse_scale_shift_raw, dit_group_norm_silu_noalloc_raw, dit_group_norm_silu_raw,
    fuse_scale_shift, fuse_scale_shift_backward, group_norm_silu, group_norm_silu_schedule,
    group_norm_silu_workspace_size, kernel_info, layer_norm, layer_norm_backward,
    layer_norm_backward_workspace_size, load_library, qknorm_rope_backward,
    qknorm_rope_backward_workspace_size, qknorm_rope_fused, qknorm_rope_fused_raw, strerror,
    version,
)

__all__ = ["qknorm_rope_fused", "qknorm_rope_fused_raw", "fuse_scale_shift",
           "dit_fuse_scale_shift_raw", "group_norm_silu", "group_norm_silu_schedule",
           "group_norm_silu_workspace_size",
           "dit_group_norm_silu_raw", "dit_group_norm_silu_noalloc_raw", "kernel_info",
           "attention", "attention_backward", "attention_workspace_size",
           "layer_norm", "layer_norm_backward", "layer_norm_backward_workspace_size",
           "fuse_scale_shift_backward", "qknorm_rope_backward",
           "qknorm_rope_backward_workspace_size",
           "load_library", "strerror", "version",
           "QkrError", "EXPORTS", "LIB_PATH"]
