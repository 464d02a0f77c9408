"""MI355X-native retention operator: chunkwise and parallel forward, backward, decode step, gated
variants, and the gated retention layer around it; and the operators that stand around a mixer in
a block: layer normalisation, rotary positions, the short causal convolution and the selective scan.

The operator runs in libretention_fwd.so (hand-written HIP kernels for gfx950) behind
the C ABI in include/retention.h; this package is its Python binding.  Importing the
package does not load the library; the first call does, and raises if it is missing.
"""
from ._block import (  # noqa: F401
    causal_conv_bwd,
    causal_conv_fwd,
    causal_conv_step,
    layer_norm_bwd,
    layer_norm_fwd,
    rotary_bwd,
    rotary_frequencies,
    rotary_fwd,
    rotary_table,
    scan_bwd_workspace_bytes,
    scan_workspace_bytes,
    selective_scan_bwd,
    selective_scan_fwd,
    selective_scan_step,
)
from ._lib import (  # noqa: F401
    RetentionError,
    bwd_workspace_bytes,
    calib_mfma,
    gated_msr_fwd,
    gated_retention_chunkwise_bwd,
    gated_retention_chunkwise_fwd,
    gated_retention_decode_step,
    gated_retention_parallel_fwd,
    lib,
    msr_workspace_bytes,
    profile_enable,
    profile_read,
    retention_chunkwise_bwd,
    retention_chunkwise_fwd,
    retention_chunkwise_fwd_noalloc,
    retention_decode_step,
    retention_parallel_fwd,
    workspace_bytes,
)

__all__ = [
    "retention_chunkwise_fwd",
    "retention_chunkwise_bwd",
    "gated_retention_chunkwise_bwd",
    "bwd_workspace_bytes",
    "gated_retention_chunkwise_fwd",
    "retention_decode_step",
    "gated_retention_decode_step",
    "retention_parallel_fwd",
    "gated_retention_parallel_fwd",
    "workspace_bytes",
    "gated_msr_fwd",
    "msr_workspace_bytes",
    "RetentionError",
    "lib",
    "profile_enable",
    "profile_read",
    "calib_mfma",
    "retention_chunkwise_fwd_noalloc",
    "causal_conv_bwd",
    "causal_conv_fwd",
    "causal_conv_step",
    "layer_norm_bwd",
    "layer_norm_fwd",
    "rotary_bwd",
    "rotary_frequencies",
    "rotary_fwd",
    "rotary_table",
    "scan_bwd_workspace_bytes",
    "scan_workspace_bytes",
    "selective_scan_bwd",
    "selective_scan_fwd",
    "selective_scan_step",
]
