"""GPU edges of the gated linear scan: decay gates that are nearly closed or open, infinities and NaN under documents,
codes of the largest values. Inputs, tolerances and the oracle are those of tests/test_gpu_scan.py; what a
test allows beyond them stands at it.
"""
import numpy as np
import pytest
import torch

import dynamic_short_convolution_amd as dc
from oracle import held8, scan_bwd, scan_fwd
from tests.parity import to64
from tests.scan_bounds import U, bwd_bounds, fwd_bound
from tests.test_gpu_scan import TD, inputs, near

pytestmark = pytest.mark.gpu

GRADS = ("dx", "ddecay", "drate", "dgate", "dstate")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    yield
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------------
# 1 - a^2 below the smallest normal value
# ---------------------------------------------------------------------------------

# 1 - a^2 = 2 rate sigmoid(decay) there; below 2^-126 it counts as 0, so b is off by at most 2^-63, and so is
# sigmoid(decay) rate / b <= 2^-63 of ddecay's second term
B_OFF = 2.0**-63


def nearly_closed(dtype):
    s, dy, dlast = inputs(2, 7, 42, dtype, True, 0, True, seed=300)
    # decays of -88 to -82 at four rates, and ordinary ones at rates about 2^-126
    s["rate"][:28] = torch.tensor([0.1, 1e-2, 1e-3, 1e-6]).repeat_interleave(7).cuda()
    s["rate"][28:] = torch.tensor([1e-38, 3e-39] * 7).cuda()
    s["decay"][:, :, :28] = (-88.0 + torch.arange(7)).repeat(4).to(TD[dtype]).cuda()
    s["state"][0] = 0.0
    return s, dy, dlast


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_nearly_closed_decay_gates_in_steps(dtype):
    s, _, _ = nearly_closed(dtype)
    args, state = tuple(to64(s[n]) for n in ("x", "decay", "rate", "gate")), to64(s["state"])
    ry, rlast = scan_fwd(*args, None, state)
    bound = fwd_bound(*args, None, state) + np.cumsum(np.abs(args[0]), 1) * B_OFF
    y, last = dc.dynconv_scan_fwd(**s, want_state=True)
    near("y", y, ry, bound)
    near("state", last, rlast, bound[:, -1])
    st = s["state"].clone()
    for t in range(s["x"].shape[1]):
        y = dc.dynconv_scan_step(s["x"][:, t], s["decay"][:, t], s["rate"], st, gate=s["gate"][:, t])
        near(f"token {t}", y, ry[:, t], bound[:, t])
    near("state after the steps", st, rlast, bound[:, -1])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kept", ["states", "nothing", "8 bits"])
def test_nearly_closed_decay_gates_backward(kept, dtype):
    s, dy, dlast = nearly_closed(dtype)
    rate, state = to64(s["rate"]), to64(s["state"])
    x, decay, gate = (to64(s[n]) for n in ("x", "decay", "gate"))
    given = dict(s)
    if kept == "states":
        given["chunks"] = dc.dynconv_scan_fwd(**s, want_chunks=True)[1]
    elif kept == "8 bits":
        given.update({n: dc.dynconv_pack8(s[n]) for n in ("x", "decay", "gate")})
        x, decay, gate = held8(x), held8(decay), held8(gate)
    got = dc.dynconv_scan_bwd(**given, dy=dy, dstate_out=dlast, need_dstate=True)
    for name, g in zip(GRADS, got):
        assert bool(torch.isfinite(g).all()), name
    rest = (to64(dy), None, state, to64(dlast))
    ref, bounds = scan_bwd(x, decay, rate, gate, *rest), bwd_bounds(x, decay, rate, gate, *rest)
    up = np.abs(to64(dy)).sum(1, keepdims=True) + np.abs(to64(dlast))[:, None]  # at least |dh|
    for i, extra in ((0, up), (1, up * np.abs(x)), (3, up * np.abs(x)), (4, 0.0)):
        near(GRADS[i], got[i], ref[i], bounds[i] + 1.01 * extra * B_OFF)
    # drate's terms sqrt(sigmoid / (2 rate)) dh sg x of such tokens: below 2^-63 / rate
    lim = (up * np.abs(x)).sum((0, 1)) * B_OFF / rate
    near("drate", got[2][:28], ref[2][:28], bounds[2][:28] + lim[:28])
