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


# ---------------------------------------------------------------------------------
# NaN and infinities with documents
# ---------------------------------------------------------------------------------


def with_documents(B, T, D, dtype, starts, seed, scale=1.0):
    s, dy, dlast = inputs(B, T, D, dtype, True, 0, True, seed=seed)
    seq = torch.zeros(B, T, dtype=torch.int32)
    for t in starts:
        seq[:, t:] += 1
    s["seq_idx"] = seq.cuda()
    s["rate"] *= scale
    return s, dy, dlast


def both(s, dy, dlast):
    y, last, chunks = dc.dynconv_scan_fwd(**s, want_state=True, want_chunks=True)
    kw = dict(dy=dy, dstate_out=dlast, need_dstate=True)
    return (y, last), [dc.dynconv_scan_bwd(**s, chunks=c, **kw) for c in (chunks, None)]


# one and two channels per lane (runs of 16 and 8 tokens); cut into segments, or too many workgroups for that
SHAPES = [("f32", 1, 600, 70), ("bf16", 1, 600, 70), ("bf16", 1, 600, 65), ("f16", 140, 300, 64), ("f32", 140, 300, 64)]


@pytest.mark.parametrize("dtype,B,T,D", SHAPES, ids=str)
@pytest.mark.parametrize("start,end,at", [(146, 290, 148), (144, 290, 151), (128, 290, 135), (36, 290, 40), (146, 150, 148), (130, 146, 145),
                                          (146, 290, 146), (256, 290, 257)])
def test_nan_in_the_run_of_its_documents_start(dtype, B, T, D, start, end, at):
    """Nothing of it reaches another document or channel, forwards or backwards, kept states or none."""
    s, dy, dlast = with_documents(B, T, D, dtype, (start, end), 310)
    clean, cg = both(s, dy, dlast)
    hit = torch.zeros(B, T, D, dtype=torch.bool, device="cuda")
    hit[0, start:end, 5] = True
    for t in (s["x"], s["decay"], s["gate"], dy):
        keep = t[0, at, 5].clone()
        t[0, at, 5] = float("nan")
        (y, last), grads = both(s, dy, dlast)
        t[0, at, 5] = keep
        assert torch.equal(y[~hit], clean[0][~hit]) and torch.equal(last, clean[1])
        for got, want in zip(grads, cg):
            for i in (0, 1, 3):
                assert torch.equal(got[i][~hit], want[i][~hit]), GRADS[i]
            assert torch.equal(got[4], want[4])
            assert torch.equal(got[2][:5], want[2][:5]) and torch.equal(got[2][6:], want[2][6:])


@pytest.mark.parametrize("dtype,B,T,D", SHAPES, ids=str)
@pytest.mark.parametrize("documents", [True, False])
def test_infinity_stays_through_its_document(dtype, B, T, D, documents):
    """Decays of about a half, whose product over a tile underflows to zero: the state behind an infinity is not finite
    to the document's end, the gradients before one not from its start, with document ids and without."""
    starts, at = (20, 290), 33
    s, dy, dlast = with_documents(B, T, D, dtype, starts, 320, scale=6.0)
    s["rate"] = torch.clamp(s["rate"], 1.0, 4.0)
    assert 0.0 < float(torch.exp(-s["rate"].max())) < 0.1
    first, end = starts
    if not documents:
        s["seq_idx"], first, end = None, 0, T
    s["x"][0, at, 5] = float("inf")
    (y, last), grads = both(s, dy, dlast)
    assert not bool(torch.isfinite(y[0, at:end, 5]).any())
    assert bool(torch.isfinite(last[0, 5])) == documents
    for g in grads:  # through h_{t-1}
        assert not bool(torch.isfinite(g[1][0, at + 1:end, 5]).any()) and not bool(torch.isfinite(g[2][5]))
    s["x"][0, at, 5] = 1.0
    back = end - 7
    dy[0, back, 5] = float("inf")
    for g in both(s, dy, dlast)[1]:
        assert not bool(torch.isfinite(g[0][0, first:back + 1, 5]).any())
        assert bool(torch.isfinite(g[4][0, 5])) == documents


# ---------------------------------------------------------------------------------
# Codes of the largest values
# ---------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 65])
def test_codes_of_values_past_2_to_127(dtype, D):
    """Their steps are 2^121, 128 of which no float32 holds."""
    s, dy, dlast = inputs(2, 40, D, dtype, True, 0, True, seed=330)
    s["x"][0, 3, 7], s["x"][1, 9, 11] = 1.5 * 2.0**127, -1.25 * 2.0**127
    s["gate"][0, 3, 7] = s["gate"][1, 9, 11] = -9.0
    s["decay"][0, 11, 9], s["decay"][1, 30, 2], s["decay"][1, 31, 2] = 1.5 * 2.0**127, -1.5 * 2.0**127, 2.0**127
    s["gate"][1, 20, 1], s["gate"][0, 20, 1] = 1.75 * 2.0**127, -1.0 * 2.0**127
    dy = dy * 2.0**-20
    dlast = dlast * 2.0**-20
    packed = {n: dc.dynconv_pack8(s[n]) for n in ("x", "decay", "gate")}
    held = [held8(to64(s[n])) for n in ("x", "decay", "gate")]
    args = (held[0], held[1], to64(s["rate"]), held[2])
    rest = (to64(dy), None, to64(s["state"]), to64(dlast))
    with np.errstate(over="ignore"):
        ref, bounds = scan_bwd(*args, *rest), bwd_bounds(*args, *rest)
    got = dc.dynconv_scan_bwd(**{**s, **packed}, dy=dy, dstate_out=dlast, need_dstate=True)
    for name, g, r, b in zip(GRADS, got, ref, bounds):
        near(name, g, r, b)


# ---------------------------------------------------------------------------------
# Open gates
# ---------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kept", ["whole", "8 bits"])
def test_gradients_of_open_gates(kept, dtype):
    """ddecay and dgate carry the factors 1 - sigmoid, which are small for open gates: the bounds of the others times
    them, and (|z| + 6) u of their own."""
    s, dy, dlast = inputs(2, 260, 66, dtype, True, 30, True, seed=340)
    s["decay"][:, :, :40] = torch.linspace(4.0, 20.0, 40).to(TD[dtype]).cuda()
    s["gate"][:, :, 20:] = torch.linspace(4.0, 20.0, 46).to(TD[dtype]).cuda()
    x, decay, gate = (to64(s[n]) for n in ("x", "decay", "gate"))
    given = dict(s)
    if kept == "8 bits":
        given.update({n: dc.dynconv_pack8(s[n]) for n in ("x", "decay", "gate")})
        x, decay, gate = held8(x), held8(decay), held8(gate)
    rest = (to64(dy), s["seq_idx"].cpu().numpy(), to64(s["state"]), to64(dlast))
    args = (x, decay, to64(s["rate"]), gate)
    ref, bounds = scan_bwd(*args, *rest), bwd_bounds(*args, *rest)
    got = dc.dynconv_scan_bwd(**given, dy=dy, dstate_out=dlast, need_dstate=True)
    for i, z in ((1, decay), (3, gate)):
        own = (np.abs(z) + 6) * U
        near(GRADS[i], got[i], ref[i], bounds[i] / (1.0 + np.exp(z)) * (1 + own) + own * np.abs(ref[i]))
    for i in (0, 2, 4):
        near(GRADS[i], got[i], ref[i], bounds[i])
