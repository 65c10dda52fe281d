"""MI355X (gfx950) selective-scan hot path: fused prefill scan, in-place decode
step, multi-head chunked scan and its in-place decode step, the gated delta rule
(chunked, backward, decode step), the block norm, and attention with a sliding
window and sinks (whole sequences, backward, paged cache of 8, 16 or 32 bits,
decode step), as hand-written HIP kernels behind the C ABI of include/ssm_mi355x.h.  This package is the thin Python
binding."""
from .attn import (  # noqa: F401
    attn_bwd,
    attn_cache_write,
    attn_decode_step,
    attn_fwd,
)
from .binding import (  # noqa: F401
    EXPORTED,
    Call,
    LIB_PATH,
    SCAN_BLOCKED,
    SsmError,
    chunk_decode_step,
    chunk_scan_fwd,
    decode_step,
    layer_fwd,
    lib,
    linear_fwd,
    scan_bwd,
    scan_fwd,
    scan_fwd_noalloc,
    set_timing_events,
)
from .delta import (  # noqa: F401
    block_norm_bwd,
    block_norm_fwd,
    delta_chunk_bwd,
    delta_chunk_fwd,
    delta_decode_step,
)
