"""Refusals of the gated delta rule's entry points on the host: arguments beyond test_delta_cpu.py's."""
import pytest

from tests.test_delta_cpu import (B_, BETA, BF16, DB, DG, DK_, DKN, DO, DQ, DV_, DVN, G, HK, HV, INVALID, K, O, OK, Q, S, SI, T_, V,
                                  WORKSPACE, contig, lib)  # noqa: F401


def calls(lib, eps, B=B_):  # noqa: F811
    """The statuses of the three entry points (no workspace, so nothing is launched)."""
    kk, vv, gg, st = contig(B, T_, HK, DKN), contig(B, T_, HV, DVN), contig(B, T_, HV), contig(B, HV, DKN, DVN)
    head = (Q, S(kk), K, S(kk), V, S(vv), G, S(gg), BETA, S(gg))
    tail = (B, T_, HK, HV, DKN, DVN, 0.1, eps, BF16, None, 0, None)
    yield lib.dynconv_delta_fwd(*head, None, None, None, None, O, S(vv), None, None, *tail)
    yield lib.dynconv_delta_bwd(*head, None, None, None, None, DO, S(vv), None, None, DQ, S(kk), DK_, S(kk), DV_, S(vv), DG, S(gg),
                                DB, S(gg), None, None, *tail)
    if eps != eps or B == 0:  # otherwise the step would launch
        yield lib.dynconv_delta_step(Q, S(kk[1:]), K, S(kk[1:]), V, S(vv[1:]), G, S(gg[1:]), BETA, S(gg[1:]), SI, S(st), O, S(vv[1:]),
                                     B, HK, HV, DKN, DVN, 0.1, eps, BF16, None)


@pytest.mark.parametrize("B", [B_, 0])
def test_nan_epsilon_is_refused(lib, B):  # noqa: F811
    """It is neither at least 0 (q and k normalised) nor below (as given)."""
    assert list(calls(lib, float("nan"), B)) == [INVALID] * 3


@pytest.mark.parametrize("eps", [-1.0, -float("inf"), 0.0, 1e-6, float("inf")])
def test_other_epsilons_pass(lib, eps):  # noqa: F811
    assert list(calls(lib, eps)) == [WORKSPACE] * 2
    assert list(calls(lib, eps, 0)) == [OK] * 3
