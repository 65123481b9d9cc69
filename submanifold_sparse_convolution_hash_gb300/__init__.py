"""Submanifold sparse convolution on one GB300 (sm_103a).

The compute path is libsc.so (CUDA, C ABI in include/sc.h); ``binding``
wraps it for torch tensors.  ``scenes`` draws seeded synthetic inputs.
"""
from .binding import (  # noqa: F401
    GradList,
    Hash,
    KernelMap,
    ScError,
    launch_count,
    lib,
    profile_collect,
    profile_enable,
    profile_only,
    profile_reset,
    rope_frequencies,
    sc_add_norm_bwd,
    sc_add_norm_fwd,
    sc_attn_bwd,
    sc_attn_check,
    sc_attn_fwd,
    sc_grad_clip,
    sc_hash_build,
    sc_hash_build_conv_out,
    sc_kmap_build,
    sc_kmap_build_conv,
    sc_linear_bwd,
    sc_linear_fwd,
    sc_qk_norm_rope_bwd,
    sc_qk_norm_rope_fwd,
    sc_rows_check,
    sc_subm_conv_bwd_data,
    sc_subm_conv_bwd_weight,
    sc_subm_conv_fwd,
    sc_subm_conv_tune,
)
