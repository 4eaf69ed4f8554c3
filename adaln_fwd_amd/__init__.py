"""Fused AdaLN (LayerNorm-Modulate) forward and backward for AMD Instinct
MI355X (gfx950), as hand-written HIP kernels behind a C ABI
(include/adaln.h).  PyTorch supplies device memory and streams only."""

from ._lib import AdalnError, BF16, F32, LIB_PATH, load
from .ops import (SegTable, bshape, bwd, bwd_dmod, bwd_dx, bwd_finish,
                  bwd_fused, bwd_fused_plan, bwd_noalloc, bwd_segments,
                  bwd_segments_workspace_bytes, bwd_workspace_bytes, fwd,
                  fwd_segments, max_d, plan)
from .experts import (experts_join_bwd, experts_join_fwd, experts_plan,
                      experts_plan_workspace_bytes, experts_sort_bwd,
                      experts_sort_fwd)
from .glu import glu_bwd, glu_bwd_workspace_bytes, glu_fwd
from .heads import (qk_norm_rope_bwd, qk_norm_rope_bwd_workspace_bytes,
                    qk_norm_rope_fwd, rope_bwd, rope_fwd, rope_freqs)
from .lin_attn import (lin_attn_bwd, lin_attn_bwd_workspace_bytes,
                       lin_attn_fwd, lin_attn_states_bytes, lin_attn_step)
from .residual import (residual_bwd, residual_bwd_segments,
                       residual_bwd_segments_workspace_bytes,
                       residual_bwd_workspace_bytes, residual_fwd,
                       residual_fwd_segments)

__all__ = ["AdalnError", "BF16", "F32", "LIB_PATH", "SegTable", "load",
           "bshape", "bwd", "bwd_dmod", "bwd_dx", "bwd_finish", "bwd_fused",
           "bwd_fused_plan", "bwd_noalloc", "bwd_segments", "bwd_segments_workspace_bytes",
           "bwd_workspace_bytes", "experts_join_bwd", "experts_join_fwd",
           "experts_plan", "experts_plan_workspace_bytes", "experts_sort_bwd",
           "experts_sort_fwd", "fwd", "fwd_segments", "glu_bwd",
           "glu_bwd_workspace_bytes", "glu_fwd", "lin_attn_bwd",
           "lin_attn_bwd_workspace_bytes", "lin_attn_fwd",
           "lin_attn_states_bytes", "lin_attn_step", "max_d", "plan", "qk_norm_rope_bwd",
           "qk_norm_rope_bwd_workspace_bytes", "qk_norm_rope_fwd", "residual_bwd",
           "residual_bwd_segments", "residual_bwd_segments_workspace_bytes",
           "residual_bwd_workspace_bytes", "residual_fwd",
           "residual_fwd_segments", "rope_bwd",
           "rope_fwd", "rope_freqs"]
