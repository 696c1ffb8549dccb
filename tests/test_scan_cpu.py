"""The gated linear scan, the group norm and the 8-bit activations on the host: pins of their float64 oracle, and
every validation path of their C entry points and bindings (statuses come before any HIP call, so
these run without a GPU; device pointers below are fake and must not be touched).
"""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import dynamic_short_convolution_amd as dc
from dynamic_short_convolution_amd import _lib, build
from oracle import groupnorm_bwd, groupnorm_fwd, held8, pack8, scan_bwd, scan_fwd

OK, INVALID, UNSUP, WORKSPACE = 0, 1, 2, 3
F32, BF16, F16 = 0, 1, 2
REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rnd(seed, *shape, scale=1.0):
    return scale * np.random.default_rng(seed).standard_normal(shape)


# ---------------------------------------------------------------------------------
# Oracle pins
# ---------------------------------------------------------------------------------


def test_scan_by_hand():
    """decay of 0 halves the rate: a = e^-1 with rate 2; gate of 0 halves the input."""
    x = np.array([3.0, 5.0]).reshape(1, 2, 1)
    z = np.zeros((1, 2, 1))
    a, b = np.exp(-1.0), np.sqrt(1 - np.exp(-2.0))
    y, last = scan_fwd(x, z, np.array([2.0]), z, None, np.array([[4.0]]))
    h1 = a * 4.0 + b * 0.5 * 3.0
    h2 = a * h1 + b * 0.5 * 5.0
    np.testing.assert_allclose(y.ravel(), [h1, h2], rtol=1e-14)
    np.testing.assert_allclose(last.ravel(), [h2], rtol=1e-14)
    # without a gate the input is taken whole; a document start forgets
    y, _ = scan_fwd(x, z, np.array([2.0]), None, np.array([[7, 9]]), np.array([[4.0]]))
    np.testing.assert_allclose(y.ravel(), [a * 4.0 + b * 3.0, b * 5.0], rtol=1e-14)


def test_scan_keeps_the_variance_of_its_input():
    """sqrt(1 - a^2): with a constant decay the output of unit noise has unit variance."""
    y, _ = scan_fwd(rnd(1, 1, 200_000, 1), np.zeros((1, 200_000, 1)), np.array([0.2]))
    assert abs(y[0, 1000:].var() - 1.0) < 0.05


def test_scan_documents_are_separate_calls():
    x, d, g, s = rnd(2, 1, 9, 3), rnd(3, 1, 9, 3), rnd(4, 1, 9, 3), rnd(5, 1, 3)
    rate, seq = np.abs(rnd(6, 3)), np.array([[4, 4, 4, 1, 1, 7, 7, 7, 7]])
    y, last = scan_fwd(x, d, rate, g, seq, s)
    state = s
    for lo, hi in ((0, 3), (3, 5), (5, 9)):
        part, end = scan_fwd(x[:, lo:hi], d[:, lo:hi], rate, g[:, lo:hi], None, state if lo == 0 else None)
        np.testing.assert_allclose(y[:, lo:hi], part, rtol=1e-12)
    np.testing.assert_allclose(last, end, rtol=1e-12)


@pytest.mark.parametrize("gated,packed", [(True, True), (False, False)])
def test_scan_gradients_are_differences(gated, packed):
    B, T, D = 2, 7, 3
    x, d, dy = rnd(10, B, T, D), rnd(11, B, T, D), rnd(12, B, T, D)
    g = rnd(13, B, T, D) if gated else None
    rate, s, ds = 0.1 + np.abs(rnd(14, D)), rnd(15, B, D), rnd(16, B, D)
    seq = np.array([[0, 0, 1, 1, 1, 2, 2], [3, 3, 3, 3, 3, 3, 3]]) if packed else None

    def loss():
        y, last = scan_fwd(x, d, rate, g, seq, s)
        return (y * dy).sum() + (last * ds).sum()

    grads = scan_bwd(x, d, rate, g, dy, seq, s, ds)
    assert (grads[3] is None) == (not gated)
    check_differences((x, d, rate, g, s), grads, loss)


def check_differences(inputs, grads, loss, h=1e-6, tol=1e-7):
    for a, got in zip(inputs, grads):
        if a is None:
            continue
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = loss()
            a[i] = keep - h
            num = (up - loss()) / (2 * h)
            a[i] = keep
            assert abs(num - got[i]) <= tol * (1 + abs(got[i])), i


def test_scan_planted_mistakes_are_seen():
    """An input scale of 1 - a instead of sqrt(1 - a^2), a decay taken from the token before, and a missing
    input gate each move the outputs."""
    x, d, g, rate = rnd(20, 1, 8, 2), rnd(21, 1, 8, 2), rnd(22, 1, 8, 2), np.array([0.5, 1.5])
    y, _ = scan_fwd(x, d, rate, g)
    assert np.abs(scan_fwd(x, np.roll(d, 1, axis=1), rate, g)[0] - y).max() > 1e-2
    assert np.abs(scan_fwd(x, d, rate)[0] - y).max() > 1e-2
    a = np.exp(-rate / (1 + np.exp(-d)))
    assert np.abs(scan_fwd(x * (1 - a) / np.sqrt(1 - a * a), d, rate, g)[0] - y).max() > 1e-2


def test_groupnorm_by_hand():
    x = np.array([[[1.0, 3.0, 10.0, 30.0]]])  # groups (1, 3): mean 2, variance 1; (10, 30): 20, 100
    np.testing.assert_allclose(groupnorm_fwd(x, 2, eps=0.0), [[[-1, 1, -1, 1]]])
    y = groupnorm_fwd(x, 2, np.array([2.0, 1, 1, 1]), np.array([0.0, 1, 0, 0]), np.full((1, 1, 4), 1.0), "silu", eps=0.0)
    silu = lambda z: z / (1 + np.exp(-z))  # noqa: E731
    np.testing.assert_allclose(y[0, 0], [silu(v) * silu(1.0) for v in (-2.0, 2.0, -1.0, 1.0)])
    # one group over two tokens of a sequence of three
    x = np.array([[[1.0, 3.0], [5.0, 7.0], [100.0, 100.0]]])
    y = groupnorm_fwd(x, 1, over="sequence", lengths=[2], eps=0.0)
    np.testing.assert_allclose(y[0], np.array([[-3, -1], [1, 3], [0, 0]]) / np.sqrt(5.0))


@pytest.mark.parametrize("over,lengths", [("token", None), ("sequence", None), ("sequence", [3, 0])])
@pytest.mark.parametrize("activation", [None, "silu"])
def test_groupnorm_gradients_are_differences(over, lengths, activation):
    x, g, dy = rnd(30, 2, 4, 6), rnd(31, 2, 4, 6), rnd(32, 2, 4, 6)
    w, b = 1 + rnd(33, 6, scale=0.2), rnd(34, 6)
    args = dict(activation=activation, over=over, lengths=lengths, eps=1e-2)
    grads = groupnorm_bwd(x, 2, dy, w, b, g, **args)
    check_differences((x, w, b, g), grads, lambda: (groupnorm_fwd(x, 2, w, b, g, **args) * dy).sum(), tol=1e-6)


def test_pack8_by_hand():
    x = np.zeros((1, 130))
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 1.0, -0.99, 1 / 128, 3 / 128  # a step of 1/64: 64, -63.36, 0.5, 1.5
    x[0, 64] = 127.9  # a step of 1: cut at 127
    x[0, 128], x[0, 129] = np.inf, 1.0
    codes, steps = pack8(x)
    assert list(codes[0, :4]) == [64, -63, 0, 2] and list(steps[0, :2]) == [1 / 64, 1.0] and codes[0, 64] == 127
    assert np.isnan(held8(x)[0, 128:]).all() and np.isfinite(held8(x)[0, :128]).all()


# ---------------------------------------------------------------------------------
# C entry points
# ---------------------------------------------------------------------------------


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


P = ctypes.c_void_p
(X, A, G, RATE, Y, SI, SO, CH, DY, DX, DA, DR, DG, DSI, DSO, SEG, WS, XC, AC, GC) = (P(0x100000 * (i + 1)) for i in range(20))
S = _lib.strides
B_, T_, D_ = 2, 70, 130
ACT = [T_ * D_, D_, 1]


def pair(p, s):
    return (p, S(s)) if p is not None else (None, None)


def sfwd(lib, x=X, xs=ACT, a=A, g=G, rate=RATE, seg=None, ss=None, si=None, sis=(D_, 1), y=Y, ys=ACT, so=None, sos=(D_, 1), ch=None, B=B_, T=T_,
         D=D_, dt=BF16, ws=None, wsb=0):
    return lib.dynconv_scan_fwd(x, S(xs), a, S(ACT), *pair(g, ACT), rate, seg, S(ss) if ss else None, *pair(si, sis), y, S(ys), *pair(so, sos),
                                ch, B, T, D, dt, ws, wsb, None)


LONG = dict(B=1, T=100_000, D=64, xs=[0, 64, 1], ys=[0, 64, 1])


@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), INVALID), (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(D=-1), INVALID), (dict(B=2**31), UNSUP), (dict(T=2**31), UNSUP),
    (dict(D=2**24 + 1), UNSUP), (dict(B=2**20, D=512), UNSUP),
    (dict(x=P(0)), INVALID), (dict(a=P(0)), INVALID), (dict(rate=P(0)), INVALID), (dict(y=P(0)), INVALID),
    (dict(x=P(X.value + 1)), UNSUP), (dict(rate=P(RATE.value + 2)), UNSUP), (dict(xs=[T_ * D_, D_, 2]), UNSUP), (dict(xs=[T_ * D_, -D_, 1]), UNSUP),
    (dict(xs=[T_ << 22, 1 << 22, 1]), UNSUP), (dict(ys=[T_ << 22, 1 << 22, 1]), UNSUP),
    (dict(ys=[0, D_, 1]), INVALID), (dict(ys=[T_ * D_, 0, 1]), INVALID),  # several tokens in one place
    (dict(y=X), INVALID), (dict(y=G), INVALID), (dict(y=P(RATE.value)), INVALID), (dict(y=CH, ch=CH), INVALID), (dict(y=SI, si=SI), INVALID),
    (dict(so=X), INVALID), (dict(so=CH, ch=CH), INVALID), (dict(ch=A), INVALID), (dict(ch=SI, si=SI), INVALID), (dict(ch=P(CH.value + 2)), UNSUP),
    (dict(seg=SEG), INVALID), (dict(seg=P(SEG.value + 2), ss=[T_, 1]), UNSUP), (dict(seg=SEG, ss=[T_, -1]), UNSUP),
    (dict(si=SI, sis=[D_, 2]), UNSUP), (dict(si=P(SI.value + 2)), UNSUP), (dict(so=SO, sos=[0, 1]), INVALID),
    (dict(si=SI, so=SI, sos=[2 * D_, 1]), INVALID),  # in place, other places
    (LONG, WORKSPACE), (dict(LONG, ws=WS, wsb=100), WORKSPACE),
    (dict(LONG, ws=P(WS.value + 4), wsb=1 << 30), UNSUP),
    (dict(B=0), OK), (dict(D=0), OK), (dict(T=0), OK), (dict(T=0, si=SI, so=SI), OK)])
def test_scan_fwd_validation(lib, kw, status):
    assert sfwd(lib, **kw) == status


def sbwd(lib, x=X, a=A, g=G, xc=None, ac=None, gc=None, rate=RATE, si=None, ch=None, dy=DY, dys=ACT, dso=None, dx=DX, dxs=ACT, da=DA, dr=DR, dg=DG,
         dsi=None, dsis=(D_, 1), T=T_, ws=None, wsb=0, scs=(T_ * 3, 3, 1)):
    return lib.dynconv_scan_bwd(x, S(ACT), a, S(ACT), *pair(g, ACT), *pair(xc, scs), *pair(ac, scs), *pair(gc, scs), rate, None, None,
                                *pair(si, (D_, 1)), ch, dy, S(dys), *pair(dso, (D_, 1)), dx, S(dxs), da, S(ACT), dr, *pair(dg, ACT), *pair(dsi, dsis),
                                B_, T, D_, BF16, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=P(0)), INVALID), (dict(a=P(0)), INVALID), (dict(dy=P(0)), INVALID), (dict(dx=P(0)), INVALID), (dict(da=P(0)), INVALID),
    (dict(dr=P(0)), INVALID), (dict(rate=P(0)), INVALID), (dict(dg=None), INVALID), (dict(g=None), INVALID),  # a gate and its gradient go together
    (dict(dx=X), INVALID), (dict(da=DX), INVALID), (dict(dg=DY), INVALID), (dict(dr=RATE), INVALID), (dict(dsi=SI, si=SI), INVALID),
    (dict(dsi=DSO, dso=DSO), INVALID), (dict(dx=CH, ch=CH), INVALID), (dict(dx=XC, xc=XC, ac=AC, gc=GC), INVALID),
    (dict(xc=XC), INVALID), (dict(xc=XC, ac=AC), INVALID), (dict(ac=AC), INVALID), (dict(gc=GC), INVALID),  # all packed or none
    (dict(xc=XC, ac=AC, gc=GC, scs=(T_ * 3, 3, 2)), UNSUP), (dict(xc=XC, ac=AC, gc=GC, scs=(T_ * 3, -3, 1)), UNSUP),
    (dict(dys=[T_ << 22, 1 << 22, 1]), UNSUP), (dict(dxs=[T_ * D_, 0, 1]), INVALID), (dict(dsi=DSI, dsis=[0, 1]), INVALID),
    (dict(dr=P(DR.value + 2)), UNSUP), (dict(dy=P(DY.value + 1)), UNSUP),
    (dict(), WORKSPACE), (dict(ch=CH), WORKSPACE), (dict(xc=XC, ac=AC, gc=GC), WORKSPACE), (dict(ws=WS, wsb=100), WORKSPACE),
    (dict(ws=P(WS.value + 4), wsb=1 << 30), UNSUP)])
def test_scan_bwd_validation(lib, kw, status):
    assert sbwd(lib, **kw) == status


def sstep(lib, x=X, xs=(D_, 1), g=G, rate=RATE, st=SI, sts=(D_, 1), y=Y, ys=(D_, 1), B=B_, D=D_, dt=F16):
    return lib.dynconv_scan_step(x, S(xs), A, S((D_, 1)), *pair(g, (D_, 1)), rate, st, S(sts), y, S(ys), B, D, dt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=P(0)), INVALID), (dict(st=P(0)), INVALID), (dict(rate=P(0)), INVALID), (dict(y=P(0)), INVALID), (dict(y=X), INVALID), (dict(y=SI), INVALID),
    (dict(st=G), INVALID), (dict(dt=5), INVALID), (dict(xs=(D_, 2)), UNSUP), (dict(xs=(-D_, 1)), UNSUP), (dict(x=P(X.value + 1)), UNSUP),
    (dict(st=P(SI.value + 2)), UNSUP), (dict(sts=(0, 1)), INVALID), (dict(ys=(0, 1)), INVALID), (dict(rate=P(RATE.value + 1)), UNSUP),
    (dict(B=-1), INVALID), (dict(B=0), OK), (dict(D=0), OK)])
def test_scan_step_validation(lib, kw, status):
    assert sstep(lib, **kw) == status


def test_scan_workspace_queries(lib):
    f, b = lib.dynconv_scan_fwd_workspace_size, lib.dynconv_scan_bwd_workspace_size
    assert f(8, 4096, 2048, BF16) == 0 and f(1, 32768, 2048, BF16) > 0 and f(1, 128, 64, BF16) == 0
    for dt in (F32, BF16, F16):
        assert 0 < b(8, 4096, 2048, 1, dt) < b(8, 4096, 2048, 0, dt)
    for bad in ((-1, 5, 64), (0, 5, 64), (1, 0, 64), (1, 5, 0), (1, 2**31, 64), (2**20, 5, 512)):
        assert f(*bad, BF16) == 0 and b(*bad, 0, BF16) == 0
    assert f(1, 5, 64, 9) == 0 and b(1, 5, 64, 0, 9) == 0
    assert b(1, 2**31 - 2**17, 2**24, 0, BF16) > 2**49  # no wrap


def npack(lib, x=X, xs=(480, 160, 40, 1), c=Y, cs=(480, 160, 40, 1), s=SO, ss=(12, 4, 1, 1), n=(2, 3, 4), D=40, dt=BF16, unpack=False):
    if unpack:
        return lib.dynconv_unpack(c, S(cs), s, S(ss), x, S(xs), *n, D, dt, None)
    return lib.dynconv_pack(x, S(xs), c, S(cs), s, S(ss), *n, D, dt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=P(0)), INVALID), (dict(c=P(0)), INVALID), (dict(s=P(0)), INVALID), (dict(c=X), INVALID), (dict(s=X), INVALID), (dict(s=Y), INVALID),
    (dict(dt=8), INVALID), (dict(n=(2, -3, 4)), INVALID), (dict(D=-1), INVALID), (dict(D=2**24 + 1), UNSUP), (dict(n=(2**20, 2**11, 1)), UNSUP),
    (dict(n=(2**40, 1, 1)), UNSUP), (dict(x=P(X.value + 1)), UNSUP), (dict(xs=(480, 160, 40, 2)), UNSUP), (dict(xs=(480, -160, 40, 1)), UNSUP),
    (dict(D=100, ss=(12, 4, 1, 2)), UNSUP), (dict(n=(0, 3, 4)), OK), (dict(D=0), OK)])
@pytest.mark.parametrize("unpack", [False, True])
def test_pack_validation(lib, kw, status, unpack):
    assert npack(lib, unpack=unpack, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(cs=(480, 0, 40, 1)), INVALID), (dict(ss=(0, 4, 1, 1)), INVALID), (dict(unpack=True, xs=(0, 160, 40, 1)), INVALID)])
def test_pack_output_validation(lib, kw, status):
    assert npack(lib, **kw) == status


GACT = [T_ * 128, 128, 1]


def gfwd(lib, x=X, xs=GACT, w=A, b=RATE, g=G, ln=None, y=Y, ys=GACT, st=None, B=B_, T=T_, C=128, groups=4, seq=0, eps=1e-5, dt=BF16, ws=None, wsb=0):
    return lib.dynconv_groupnorm_fwd(x, S(xs), w, b, *pair(g, GACT), ln, y, S(ys), st, B, T, C, groups, seq, 1, eps, dt, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), INVALID), (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(C=-4), INVALID), (dict(groups=0), INVALID), (dict(groups=3), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(C=2**19 + 4), UNSUP), (dict(B=2**23), UNSUP), (dict(T=2**31), UNSUP),
    (dict(B=2**16, T=2**16), UNSUP), (dict(x=P(0)), INVALID), (dict(y=P(0)), INVALID), (dict(y=X), INVALID), (dict(y=A), INVALID), (dict(y=G), INVALID),
    (dict(x=P(X.value + 1)), UNSUP), (dict(w=P(A.value + 1)), UNSUP), (dict(xs=[T_ * 128, 128, 2]), UNSUP), (dict(xs=[-1, 128, 1]), UNSUP),
    (dict(ys=[T_ * 128, 0, 1]), INVALID), (dict(ln=SEG), INVALID), (dict(st=SO), INVALID),  # over sequences only
    (dict(seq=1, ln=P(SEG.value + 2)), UNSUP), (dict(seq=1, st=P(SO.value + 1)), UNSUP), (dict(seq=1, st=X), INVALID), (dict(seq=1, st=Y), INVALID),
    (dict(seq=1, ln=SEG), WORKSPACE), (dict(seq=1, st=SO), WORKSPACE), (dict(seq=1, ws=P(WS.value + 4), wsb=1 << 30), UNSUP),
    (dict(B=0), OK), (dict(T=0), OK), (dict(C=0), OK)])
def test_groupnorm_fwd_validation(lib, kw, status):
    assert gfwd(lib, **kw) == status


def gbwd(lib, x=X, xc=None, xcs=(T_ * 2, 2, 1), w=A, g=G, ln=None, st=None, dy=DY, dx=DX, dxs=GACT, dw=DR, db=DA, dg=DG, seq=0, ws=None, wsb=0, T=T_):
    return lib.dynconv_groupnorm_bwd(x, S(GACT), *pair(xc, xcs), w, RATE, *pair(g, GACT), ln, st, dy, S(GACT), dx, S(dxs), dw, db, *pair(dg, GACT),
                                     B_, T, 128, 4, seq, 0, 1e-5, BF16, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=P(0)), INVALID), (dict(dy=P(0)), INVALID), (dict(dx=P(0)), INVALID), (dict(dg=None), INVALID), (dict(g=None), INVALID),
    (dict(dx=X), INVALID), (dict(dx=DY), INVALID), (dict(db=DR), INVALID), (dict(dw=A), INVALID), (dict(dg=DX), INVALID), (dict(dx=XC, xc=XC), INVALID),
    (dict(xc=XC, xcs=(T_ * 2, 2, 2)), UNSUP), (dict(xc=XC, xcs=(T_ * 2, -2, 1)), UNSUP), (dict(dw=P(DR.value + 2)), UNSUP),
    (dict(dxs=[0, 128, 1]), INVALID), (dict(ln=SEG), INVALID), (dict(st=SO), INVALID), (dict(seq=1, ln=P(SEG.value + 1)), UNSUP),
    (dict(), WORKSPACE), (dict(seq=1, dw=None, db=None), WORKSPACE), (dict(seq=1, st=SO), WORKSPACE), (dict(ws=P(WS.value + 4), wsb=1 << 30), UNSUP)])
def test_groupnorm_bwd_validation(lib, kw, status):
    assert gbwd(lib, **kw) == status


def test_groupnorm_workspace_queries(lib):
    f, b = lib.dynconv_groupnorm_fwd_workspace_size, lib.dynconv_groupnorm_bwd_workspace_size
    assert f(8, 4096, 2048, 16, 0, 0, BF16) == 0 < f(8, 4096, 2048, 16, 1, 1, BF16) < f(8, 4096, 2048, 16, 1, 0, BF16)
    assert 0 < b(8, 4096, 2048, 16, 0, 0, BF16) and 0 < b(8, 4096, 2048, 16, 1, 1, BF16) < b(8, 4096, 2048, 16, 1, 0, BF16)
    for bad in ((-1, 5, 64, 4), (0, 5, 64, 4), (1, 0, 64, 4), (1, 5, 0, 4), (1, 5, 64, 5), (1, 5, 64, 0), (1, 2**31, 64, 4), (2**16, 2**16, 64, 4)):
        for seq in (0, 1):
            assert f(*bad, seq, 0, BF16) == 0 and b(*bad, seq, 0, BF16) == 0
    assert b(2**23 - 1, 255, 2**19, 1, 1, 0, F32) > 2**40  # no wrap


# ---------------------------------------------------------------------------------
# Bindings
# ---------------------------------------------------------------------------------


def test_scan_binding_checks():
    x, rate, st = torch.zeros(2, 3, 8), torch.ones(8), torch.zeros(2, 8)
    for kw in (dict(gate=x[:1]), dict(state=st[:1]), dict(state_out=torch.zeros(2, 9)), dict(out=x[0]), dict(seq_idx=torch.zeros(2, 4, dtype=torch.int32)),
               dict(seq_idx=torch.zeros(2, 3))):
        with pytest.raises((ValueError, RuntimeError)):
            dc.dynconv_scan_fwd(x, x, rate, **kw)
    for bad in (dict(decay=x[..., :4]), dict(decay=None), dict(rate=torch.ones(7)), dict(rate=torch.ones(16)[::2]), dict(rate=None)):
        with pytest.raises(ValueError):
            dc.dynconv_scan_fwd(**{**dict(x=x, decay=x, rate=rate), **bad})
    for bad in (dict(decay=x.half()), dict(rate=rate.double()), dict(x=x.double(), decay=x.double())):
        with pytest.raises(TypeError):
            dc.dynconv_scan_fwd(**{**dict(x=x, decay=x, rate=rate), **bad})
    with pytest.raises(ValueError):
        dc.dynconv_scan_fwd(x[0], x[0], rate)
    packed = dc.Packed8(torch.zeros(2, 3, 8, dtype=torch.int8), torch.zeros(2, 3, 1, dtype=torch.uint8))
    for kw in (dict(x=packed), dict(decay=packed), dict(gate=packed), dict(x=packed, decay=packed, gate=x), dict(dy=x[:1]), dict(chunks=torch.zeros(2, 2, 8)),
               dict(chunks=torch.zeros(2, 1, 16)[..., ::2]), dict(dstate_out=st[:1]),
               dict(x=packed._replace(scales=packed.scales[:1]), decay=packed), dict(x=packed._replace(codes=packed.codes[:1]), decay=packed)):
        with pytest.raises(ValueError):
            dc.dynconv_scan_bwd(**{**dict(x=x, decay=x, rate=rate, dy=x), **kw})
    with pytest.raises(TypeError):
        dc.dynconv_scan_bwd(packed._replace(codes=torch.zeros(2, 3, 8, dtype=torch.uint8)), packed, rate, x)
    with pytest.raises(ValueError, match="state"):
        dc.dynconv_scan_step(x[:, 0], x[:, 0], rate, None)
    with pytest.raises(ValueError):
        dc.dynconv_scan_step(x[:, 0], x[:, 0], rate, st[:1])
    with pytest.raises(RuntimeError, match="GPU only"):
        dc.dynconv_scan_fwd(x, x, rate)
    with pytest.raises(RuntimeError, match="GPU only"):
        dc.dynconv_scan_bwd(packed, packed, rate, x)


def test_pack8_binding_checks():
    x = torch.zeros(2, 3, 70)
    with pytest.raises(TypeError):
        dc.dynconv_pack8(x.double())
    with pytest.raises(ValueError):
        dc.dynconv_pack8(torch.zeros(1, 1, 1, 1, 8))
    with pytest.raises(ValueError):
        dc.dynconv_pack8(x, out=dc.Packed8(torch.zeros(2, 3, 70, dtype=torch.int8), torch.zeros(2, 3, 1, dtype=torch.uint8)))
    good = dc.Packed8(torch.zeros(2, 3, 70, dtype=torch.int8), torch.zeros(2, 3, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        dc.dynconv_unpack8(good._replace(scales=good.scales[..., :1]))
    with pytest.raises(TypeError):
        dc.dynconv_unpack8(good, out=x)  # bfloat16 asked for
    with pytest.raises(RuntimeError, match="GPU only"):
        dc.dynconv_pack8(x)


def test_groupnorm_binding_checks():
    x, w = torch.zeros(2, 3, 8), torch.ones(8)
    for kw in (dict(weight=w[:7]), dict(bias=torch.ones(16)[::2]), dict(gate=x[:1]), dict(out=x[0]), dict(activation="gelu"), dict(over="batch"),
               dict(groups=3), dict(groups=0), dict(lengths=torch.ones(2, dtype=torch.int32)), dict(over="sequence", lengths=torch.ones(3, dtype=torch.int32)),
               dict(over="sequence", lengths=torch.ones(4, dtype=torch.int32)[::2])):
        with pytest.raises(ValueError):
            dc.dynconv_groupnorm_fwd(**{**dict(x=x, groups=2), **kw})
    with pytest.raises(TypeError):
        dc.dynconv_groupnorm_fwd(x, 2, w.half())
    with pytest.raises(TypeError):
        dc.dynconv_groupnorm_fwd(x, 2, over="sequence", lengths=torch.ones(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        dc.dynconv_groupnorm_fwd(x[0], 2, over="sequence")
    with pytest.raises(ValueError):
        dc.dynconv_groupnorm_fwd(x[0, 0], 2)
    for kw in (dict(dy=x[:1]), dict(stats=torch.zeros(2, 2, 2)), dict(over="sequence", stats=torch.zeros(2, 4, 2)),
               dict(x=dc.Packed8(torch.zeros(2, 3, 8, dtype=torch.int8), torch.zeros(2, 3, 2, dtype=torch.uint8)))):
        with pytest.raises(ValueError):
            dc.dynconv_groupnorm_bwd(**{**dict(x=x, groups=2, dy=x), **kw})
    with pytest.raises(RuntimeError, match="GPU only"):
        dc.dynconv_groupnorm_fwd(x, 2)


def test_entry_points_under_sanitizers():
    """The validation tests above once more against the host-only build of the library with
    AddressSanitizer and UndefinedBehaviorSanitizer."""
    if os.environ.get("DYNCONV_LIBRARY"):
        pytest.skip("already the sanitized run")
    try:
        runtime = build.sanitizer_runtime()
    except RuntimeError as e:
        pytest.skip(f"no sanitizer runtime: {e}")
    from tests.test_abi_sanitized import _stale

    if _stale(build.ASAN_LIB_PATH):
        build.build_host_sanitized()
    env = dict(os.environ, LD_PRELOAD=runtime, DYNCONV_LIBRARY=build.ASAN_LIB_PATH,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    cmd = [sys.executable, "-m", "pytest", os.path.abspath(__file__), "-x", "-q", "-p", "no:cacheprovider", "-k",
           "validation or workspace or binding"]
    res = subprocess.run(cmd, cwd=REPO, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-6000:]
    assert res.returncode == 0 and " passed" in out, out[-6000:]
