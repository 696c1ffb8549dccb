"""MI355X-native dynamic short convolution: HIP kernels for gfx950 behind a C ABI.

The Python surface mirrors the C entry points of include/dynconv.h:
dynconv_fwd, dynconv_bwd, dynconv_lowrank_fwd, dynconv_lowrank_bwd (and the workspace
queries), and for inference dynconv_cache_fill, dynconv_decode_step and
dynconv_lowrank_decode_step (with new_cache for a zeroed rolling cache), and the
convolution fused into its producing projection, dynconv_gemm_fwd and
dynconv_gemm_lowrank_fwd. What consumes the convolved q, k, v in a linear-attention layer:
the gated delta rule, dynconv_delta_fwd, dynconv_delta_bwd and the decoding step
dynconv_delta_step (with new_delta_state), and the RMS norm with weight, SiLU gate and
residual, dynconv_norm_fwd and dynconv_norm_bwd. The other recurrence behind a convolution, the
gated linear scan per channel: dynconv_scan_fwd, dynconv_scan_bwd and the decoding step
dynconv_scan_step (with new_scan_state), and the group norm with weight, bias, SiLU and gate, per
token or over a sequence, dynconv_groupnorm_fwd and dynconv_groupnorm_bwd. What a training step keeps for its backward pass in 8
bits: dynconv_pack8 and dynconv_unpack8, whose Packed8 those two's backward calls read. Importing this package does not load the
library; the first call does, and fails loudly if it has not been built.
"""
from .ops import (  # noqa: F401
    dynconv_bwd,
    dynconv_bwd_workspace_size,
    dynconv_cache_fill,
    dynconv_decode_step,
    dynconv_delta_bwd,
    dynconv_delta_fwd,
    dynconv_delta_step,
    dynconv_fwd,
    dynconv_gemm_fwd,
    dynconv_gemm_lowrank_fwd,
    dynconv_groupnorm_bwd,
    dynconv_groupnorm_fwd,
    dynconv_lowrank_bwd,
    dynconv_lowrank_bwd_workspace_size,
    dynconv_lowrank_decode_step,
    dynconv_lowrank_fwd,
    dynconv_norm_bwd,
    dynconv_norm_fwd,
    dynconv_pack8,
    dynconv_scan_bwd,
    dynconv_scan_fwd,
    dynconv_scan_step,
    dynconv_unpack8,
    new_cache,
    new_delta_state,
    new_scan_state,
    Packed8,
)
from ._lib import DynconvError, load  # noqa: F401
