"""Placement-aware gradient reduction, global norm, clipping and fused AdamW
for MI355X (gfx950): a C-ABI library of hand-written HIP kernels
(libgro.so, declared in include/gro.h) with a thin ctypes binding.

The library is loaded on first use and there is no fallback: a missing
library raises.
"""
from .binding import (  # noqa: F401
    GroError, gro_accumulate, gro_accumulate_window, gro_clip_adamw, gro_last_error, gro_plan_bind, gro_plan_bucket,
    gro_plan_create, gro_plan_destroy, gro_plan_get_info, gro_plan_get_norm, gro_plan_tensor,
    gro_init_uniform, gro_reduce_norm, load,
    gro_clip_adamw_coded, gro_group_bind, gro_group_clip_adamw, gro_group_create, gro_group_destroy,
    gro_group_get_info, gro_group_get_norm, gro_group_norm, gro_moments_decode, gro_moments_encode,
    gro_experts_forward, gro_experts_input_grad, gro_experts_weight_grad, gro_experts_workspace, gro_lookup,
    gro_lookup_grad, gro_lookup_grad_workspace, gro_row_sort, gro_row_sort_workspace,
)
