"""MI355X (gfx950) Kimi Delta Attention: chunked prefill, its backward, and the fused recurrence;
linear attention with one decay per head in the same three forms; and the norms round such a block.

The computation lives in the HIP library ``_build/libkda.so`` (C ABI in ``include/kda.h``,
``include/kda_linear.h`` and ``include/kda_norm.h``); this package only marshals arguments to it.
"""
from ._binding import (KdaError, chunk_kda, chunk_kda_bwd, chunk_kda_noalloc, gate_cumsum, lib, recurrent_kda,  # noqa: F401
                       resolved_schedule, resolved_segment, workspace_bytes, check_offsets)
from ._linear import (block_norm, block_norm_bwd, chunk_linear_attn, chunk_linear_attn_bwd,  # noqa: F401
                      linear_workspace_bytes, recurrent_linear_attn)

__all__ = ["chunk_kda", "chunk_kda_bwd", "chunk_kda_noalloc", "recurrent_kda", "gate_cumsum", "KdaError", "lib", "resolved_schedule", "resolved_segment", "check_offsets",
           "workspace_bytes", "chunk_linear_attn", "chunk_linear_attn_bwd", "recurrent_linear_attn",
           "linear_workspace_bytes", "block_norm", "block_norm_bwd"]
