"""Refusals of the gated linear scan and the group norm that take 8-bit inputs together with what the forward kept of
others, at the C entry points and in the bindings (no GPU: statuses come before any HIP call).
"""
import pytest
import torch

import dynamic_short_convolution_amd as dc
from tests.test_scan_cpu import AC, CH, GC, INVALID, SO, XC, WORKSPACE, gbwd, lib, sbwd  # noqa: F401


def test_scan_kept_states_do_not_go_with_codes(lib):  # noqa: F811
    assert sbwd(lib, xc=XC, ac=AC, gc=GC) == WORKSPACE  # nothing else is missing
    assert sbwd(lib, xc=XC, ac=AC, gc=GC, ch=CH) == INVALID
    assert sbwd(lib, xc=XC, ac=AC, g=None, dg=None, ch=CH) == INVALID
    x, rate = torch.zeros(2, 3, 8), torch.ones(8)
    packed = dc.Packed8(torch.zeros(2, 3, 8, dtype=torch.int8), torch.zeros(2, 3, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="chunks"):
        dc.dynconv_scan_bwd(packed, packed, rate, x, chunks=torch.zeros(2, 1, 8))


def test_groupnorm_statistics_do_not_go_with_codes(lib):  # noqa: F811
    assert gbwd(lib, xc=XC, seq=1) == WORKSPACE
    assert gbwd(lib, xc=XC, seq=1, st=SO) == INVALID
    packed = dc.Packed8(torch.zeros(2, 3, 8, dtype=torch.int8), torch.zeros(2, 3, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="stats"):
        dc.dynconv_groupnorm_bwd(packed, 2, torch.zeros(2, 3, 8), over="sequence", stats=torch.zeros(2, 2, 2))
