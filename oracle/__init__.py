"""float64 CPU oracle of the dynamic short convolution, and of the gated delta rule and gated
norm that consume its outputs, the gated linear scan, the group norm and activations in 8 bits
(test infrastructure only).

Used by the tests, the package smoke check and the benchmark's CPU-baseline leg; never
by the product path. See ``dynconv_oracle``, ``delta_oracle`` and ``scan_oracle`` for what they compute and where it comes from.
"""
from .delta_oracle import delta_bwd, delta_fwd, norm_bwd, norm_fwd  # noqa: F401
from .dynconv_oracle import (  # noqa: F401
    conv_bias_grad,
    conv_bwd,
    conv_fwd,
    gemm_conv_fwd,
    gemm_lowrank_fwd,
    lowrank_bwd,
    lowrank_filters,
    lowrank_fwd,
    projection,
)
from .scan_oracle import groupnorm_bwd, groupnorm_fwd, held8, linear_scan, pack8, scan_bwd, scan_fwd, scan_terms  # noqa: F401
