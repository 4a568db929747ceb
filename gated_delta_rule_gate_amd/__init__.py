"""MI355X (gfx950) Kimi Delta Attention: chunked prefill, its backward, and the fused recurrence;
the gated delta rule and linear attention with one decay per head in the same three forms; the norm
and rotation of their query and key rows; and the norms round such a block.

The computation lives in the HIP library ``_build/libkda.so`` (C ABI in ``include/kda.h``,
``include/kda_delta.h``, ``include/kda_linear.h``, ``include/kda_rope.h`` and ``include/kda_norm.h``); this package only marshals arguments to it.
"""
from ._binding import (KdaError, chunk_kda, chunk_kda_bwd, chunk_kda_noalloc, gate_cumsum, lib, recurrent_kda,  # noqa: F401
                       resolved_schedule, resolved_segment, workspace_bytes, check_offsets)
from ._delta import (chunk_gated_delta, chunk_gated_delta_bwd, gated_delta_workspace_bytes, qk_norm_rope,  # noqa: F401
                     qk_norm_rope_bwd, recurrent_gated_delta)
from ._linear import (block_norm, block_norm_bwd, chunk_linear_attn, chunk_linear_attn_bwd,  # noqa: F401
                      linear_workspace_bytes, recurrent_linear_attn)

__all__ = ["chunk_kda", "chunk_kda_bwd", "chunk_kda_noalloc", "recurrent_kda", "gate_cumsum", "KdaError", "lib", "resolved_schedule", "resolved_segment", "check_offsets",
           "workspace_bytes", "chunk_linear_attn", "chunk_linear_attn_bwd", "recurrent_linear_attn",
           "linear_workspace_bytes", "block_norm", "block_norm_bwd", "chunk_gated_delta", "chunk_gated_delta_bwd",
           "recurrent_gated_delta", "gated_delta_workspace_bytes", "qk_norm_rope", "qk_norm_rope_bwd"]
