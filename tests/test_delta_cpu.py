"""The gated delta rule and the gated norm on the host: pins of their float64 oracle, and every
validation path of their C entry points and bindings (statuses come before any HIP call, so
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
from oracle import delta_bwd, delta_fwd, norm_bwd, norm_fwd

OK, INVALID, UNSUP, WORKSPACE = 0, 1, 2, 3
F32, BF16, F16 = 0, 1, 2
REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rnd(seed, *shape, scale=1.0):
    return scale * np.random.default_rng(seed).standard_normal(shape)


def inputs(seed, B=1, T=5, Hk=1, Hv=2, dk=3, dv=4):
    return (rnd(seed, B, T, Hk, dk), rnd(seed + 1, B, T, Hk, dk), rnd(seed + 2, B, T, Hv, dv),
            -np.abs(rnd(seed + 3, B, T, Hv)), 1 / (1 + np.exp(-rnd(seed + 4, B, T, Hv))))


# ---------------------------------------------------------------------------------
# Oracle pins
# ---------------------------------------------------------------------------------


def test_delta_by_hand():
    """Two tokens, one head, dk = dv = 1, no normalisation: S1 = b1 v1 k1;
    S2 = a S1 + k2 b2 (v2 - a S1 k2)."""
    q, k, v = np.array([2.0, 3.0]), np.array([0.5, 2.0]), np.array([4.0, 1.0])
    g, b = np.log(np.array([0.7, 0.25])), np.array([0.5, 1.0])
    s1 = 0.5 * 0.5 * 4.0  # 1
    s2 = 0.25 * s1 + 2.0 * 1.0 * (1.0 - 0.25 * s1 * 2.0)  # 0.25 + 2 * 0.5 = 1.25
    shape = lambda a: a.reshape(1, 2, 1, 1)  # noqa: E731
    o, S = delta_fwd(shape(q), shape(k), shape(v), g.reshape(1, 2, 1), b.reshape(1, 2, 1), 0.1)
    np.testing.assert_allclose(o.ravel(), [0.1 * 2 * s1, 0.1 * 3 * s2], rtol=1e-14)
    np.testing.assert_allclose(S.ravel(), [1.25], rtol=1e-14)


def test_delta_full_write_is_interpolation():
    """beta = 1, unit orthogonal keys, no decay: the state maps each key to its value."""
    T = 4
    k = np.eye(T).reshape(1, T, 1, T)
    v = rnd(3, 1, T, 1, 6)
    o, S = delta_fwd(k, k, v, np.zeros((1, T, 1)), np.ones((1, T, 1)), 1.0)
    np.testing.assert_allclose(S[0, 0], v[0, :, 0], rtol=1e-13)
    np.testing.assert_allclose(o, v, rtol=1e-13)


def test_delta_without_erasing_is_linear_attention():
    """With orthogonal keys u_t = beta v_t: o_t = scale sum_j decay(j..t) (q_t.k_j) beta_j v_j."""
    T = 5
    q, k, v, g, b = inputs(20, T=T, Hv=1, dk=T)
    k = np.eye(T).reshape(1, T, 1, T) * rnd(7, 1, T, 1, 1)
    o, _ = delta_fwd(q, k, v, g, b, 0.3)
    G = np.cumsum(g[0, :, 0])
    for t in range(T):
        ref = sum(np.exp(G[t] - G[j]) * (q[0, t, 0] @ k[0, j, 0]) * b[0, j, 0] * v[0, j, 0] for j in range(t + 1))
        np.testing.assert_allclose(o[0, t, 0], 0.3 * ref, rtol=1e-11, atol=1e-13)


def test_delta_documents_are_separate_calls():
    q, k, v, g, b = inputs(30, T=9)
    seq = np.array([[4, 4, 4, 1, 1, 7, 7, 7, 7]])
    S0 = rnd(50, 1, 2, 3, 4)
    o, S = delta_fwd(q, k, v, g, b, 0.5, 1e-6, seq, S0)
    state = S0
    for lo, hi in ((0, 3), (3, 5), (5, 9)):
        part, state = delta_fwd(*(a[:, lo:hi] for a in (q, k, v, g, b)), 0.5, 1e-6, None, state if lo == 0 else None)
        np.testing.assert_allclose(o[:, lo:hi], part, rtol=1e-12)
    np.testing.assert_allclose(S, state, rtol=1e-12)


@pytest.mark.parametrize("eps", [None, 1e-3])
@pytest.mark.parametrize("packed", [False, True])
def test_delta_gradients_are_differences(eps, packed):
    """Central differences in every input; the map is smooth, step 1e-5: error about 1e-10."""
    args = list(inputs(40, T=6, Hk=1, Hv=2))
    seq = np.array([[0, 0, 1, 1, 1, 2]]) if packed else None
    S0, do, dS1 = rnd(60, 1, 2, 3, 4), rnd(61, 1, 6, 2, 4), rnd(62, 1, 2, 3, 4)

    def loss(*a):
        o, S = delta_fwd(*a[:5], 0.4, eps, seq, a[5])
        return np.sum(o * do) + np.sum(S * dS1)

    args.append(S0)
    grads = delta_bwd(*args[:5], do, 0.4, eps, seq, S0, dS1)
    h = 1e-5
    for a, got in zip(args, grads):
        num = np.zeros_like(a)
        it = np.nditer(a, flags=["multi_index"])
        for _ in it:
            i = it.multi_index
            keep = a[i]
            a[i] = keep + h
            up = loss(*args)
            a[i] = keep - h
            num[i] = (up - loss(*args)) / (2 * h)
            a[i] = keep
        np.testing.assert_allclose(got, num, rtol=2e-7, atol=2e-8)


def test_planted_mistakes_are_seen():
    """A decay applied after the write, a head mapping that interleaves and a missing beta in the
    erased part each move the oracle's outputs."""
    q, k, v, g, b = inputs(70, T=6, Hk=2, Hv=4)
    o, S = delta_fwd(q, k, v, g, b, 1.0)
    late, _ = delta_fwd(q, k, v, np.roll(g, 1, axis=1), b, 1.0)
    assert np.abs(late - o).max() > 1e-2
    order = [0, 2, 1, 3]  # value heads of one key head must be neighbours
    other, _ = delta_fwd(q, k, v[:, :, order], g[:, :, order], b[:, :, order], 1.0)
    assert np.abs(other[:, :, order] - o).max() > 1e-2
    scaled, _ = delta_fwd(q, k, v * b[..., None], g, np.ones_like(b), 1.0)
    assert np.abs(scaled - o).max() > 1e-2


@pytest.mark.parametrize("gated", [False, True])
def test_norm_gradients_are_differences(gated):
    x, w, z, dy = rnd(80, 3, 5), 1 + 0.2 * rnd(81, 5), rnd(82, 3, 5) if gated else None, rnd(83, 3, 5)
    got = norm_bwd(x, w, z, dy, 1e-3)
    h = 1e-6
    for a, d in zip((x, w, z), got):
        if a is None:
            assert d is None
            continue
        num = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = np.sum(norm_fwd(x, w, z, 1e-3) * dy)
            a[i] = keep - h
            num[i] = (up - np.sum(norm_fwd(x, w, z, 1e-3) * dy)) / (2 * h)
            a[i] = keep
        np.testing.assert_allclose(d, num, rtol=1e-6, atol=1e-8)


def test_norm_by_hand():
    x = np.array([[3.0, 4.0]])  # mean square 12.5
    np.testing.assert_allclose(norm_fwd(x, np.array([2.0, 1.0]), None, 0.0), [[6 / 12.5**0.5, 4 / 12.5**0.5]])
    z = np.array([[0.0, 1.0]])
    np.testing.assert_allclose(norm_fwd(x, None, z, 0.0), [[0.0, 4 / 12.5**0.5 / (1 + np.exp(-1.0))]])


# ---------------------------------------------------------------------------------
# C entry points
# ---------------------------------------------------------------------------------


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


P = ctypes.c_void_p
Q, K, V, G, BETA, SI, SO, O, DO, DQ, DK_, DV_, DG, DB, DSI, DSO, SEG, WS = (P(0x100000 * (i + 1)) for i in range(18))
S = _lib.strides
B_, T_, HK, HV, DKN, DVN = 2, 70, 2, 4, 32, 48


def contig(*shape):
    s, out = 1, []
    for n in reversed(shape):
        out.append(s)
        s *= n
    return list(reversed(out))


def fwd(lib, q=Q, qs=None, k=K, v=V, vs=None, g=G, gs=None, beta=BETA, seg=None, ss=None, si=None, sis=None, o=O, os_=None,
        so=None, sos=None, B=B_, T=T_, Hk=HK, Hv=HV, dk=DKN, dv=DVN, eps=1e-6, dt=BF16, ws=None, wsb=0):
    ks = contig(B, T, Hk, dk)
    vv = contig(B, T, Hv, dv)
    st = contig(B, Hv, dk, dv)
    return lib.dynconv_delta_fwd(
        q, S(qs or ks), k, S(ks), v, S(vs or vv), g, S(gs or contig(B, T, Hv)), beta, S(contig(B, T, Hv)), seg,
        S(ss) if ss else None, si, S(sis or st) if si else None, o, S(os_ or vv), so, S(sos or st) if so else None,
        B, T, Hk, Hv, dk, dv, 0.1, eps, dt, ws, wsb, None)


@pytest.mark.parametrize(
    "kw,status",
    [
        (dict(dt=9), INVALID),
        (dict(B=-1), INVALID),
        (dict(T=-1), INVALID),
        (dict(Hk=3), INVALID),       # 3 key heads do not divide 4 value heads
        (dict(Hk=0), INVALID),
        (dict(dk=129), UNSUP),
        (dict(dv=65537), UNSUP),
        (dict(B=2**31), UNSUP),
        (dict(T=2**31), UNSUP),
        (dict(B=2**20, Hv=2**12, Hk=1, dk=16, dv=16), UNSUP),  # more workgroups than a grid holds
        (dict(B=2**20, Hv=8, Hk=1), UNSUP),
        (dict(B=2**14, Hv=8, Hk=1, dv=32 * 64), UNSUP),
        (dict(q=P(0)), INVALID),
        (dict(v=P(0)), INVALID),
        (dict(g=P(0)), INVALID),
        (dict(o=P(0)), INVALID),
        (dict(o=V), INVALID),        # in place
        (dict(o=P(G.value)), INVALID),
        (dict(so=Q), INVALID),
        (dict(q=P(Q.value + 1)), UNSUP),  # not element aligned
        (dict(g=P(G.value + 2)), UNSUP),
        (dict(qs=[T_ * HK * DKN, HK * DKN, DKN, 2]), UNSUP),   # channels not adjacent
        (dict(qs=[T_ * HK * DKN, -HK * DKN, DKN, 1]), UNSUP),  # negative stride
        (dict(qs=[T_ << 22, 1 << 22, DKN, 1]), UNSUP),         # tokens too far apart
        (dict(os_=[T_ << 22, 1 << 22, DVN, 1]), UNSUP),
        (dict(os_=[0, HV * DVN, DVN, 1]), INVALID),            # two sequences in one place
        (dict(os_=[T_ * HV * DVN, 0, DVN, 1]), INVALID),
        (dict(seg=SEG), INVALID),                              # ids without strides
        (dict(seg=P(SEG.value + 2), ss=[T_, 1]), UNSUP),
        (dict(seg=SEG, ss=[-T_, 1]), UNSUP),
        (dict(so=SO, sos=[0, DKN * DVN, DVN, 1]), INVALID),
        (dict(si=SI, so=SI, sos=[2 * HV * DKN * DVN, DKN * DVN, DVN, 1]), INVALID),  # in place, other places
        (dict(si=P(SI.value + 2)), UNSUP),
        (dict(), WORKSPACE),
        (dict(ws=WS, wsb=1000), WORKSPACE),
        (dict(B=0), OK),
        (dict(Hv=0), OK),
        (dict(dk=0), OK),
        (dict(T=0), OK),             # no tokens and no state to write
    ],
)
def test_delta_fwd_validation(lib, kw, status):
    assert fwd(lib, **kw) == status


def bwd(lib, dO=DO, dos=None, dso=None, dq=DQ, dk_=DK_, dv_=DV_, dg=DG, db=DB, dsi=None, dqs=None, dks=None, dgs=None, dvs=None,
        ws=None, wsb=0, T=T_, si=None):
    ks, vv, gg, st = contig(B_, T_, HK, DKN), contig(B_, T_, HV, DVN), contig(B_, T_, HV), contig(B_, HV, DKN, DVN)
    return lib.dynconv_delta_bwd(
        Q, S(ks), K, S(ks), V, S(vv), G, S(gg), BETA, S(gg), None, None, si, S(st) if si else None, dO, S(dos or vv), dso,
        S(st) if dso else None, dq, S(dqs or ks), dk_, S(dks or ks), dv_, S(dvs or vv), dg, S(dgs or gg), db, S(gg), dsi,
        S(st) if dsi else None, B_, T, HK, HV, DKN, DVN, 0.1, -1.0, BF16, ws, wsb, None)


@pytest.mark.parametrize(
    "kw,status",
    [
        (dict(dO=P(0)), INVALID),
        (dict(dq=P(0)), INVALID),
        (dict(dg=P(0)), INVALID),
        (dict(db=P(0)), INVALID),
        (dict(dq=Q), INVALID),
        (dict(dk_=DQ), INVALID),     # two outputs in one place
        (dict(dv_=DO), INVALID),
        (dict(dsi=SI, si=SI), INVALID),
        (dict(dsi=DSO, dso=DSO), INVALID),
        (dict(dqs=[T_ * HK * DKN, HK * DKN, 0, 1]), INVALID),
        (dict(dgs=[T_ * HV, 0, 1]), INVALID),
        (dict(dos=[T_ << 22, 1 << 22, DVN, 1]), UNSUP),
        (dict(dvs=[T_ << 22, 1 << 22, DVN, 1]), UNSUP),
        (dict(dqs=[T_ << 22, 1 << 22, DKN, 1]), UNSUP),
        (dict(dks=[T_ << 22, 1 << 22, DKN, 1]), UNSUP),
        (dict(), WORKSPACE),
        (dict(T=0), OK),
    ],
)
def test_delta_bwd_validation(lib, kw, status):
    assert bwd(lib, **kw) == status


def step(lib, state=SI, sts=None, o=O, q=Q, dk=DKN, dt=F16, Hk=HK, os_=None):
    return lib.dynconv_delta_step(q, S(contig(B_, Hk, dk)), K, S(contig(B_, Hk, dk)), V, S(contig(B_, HV, DVN)), G,
                                  S(contig(B_, HV)), BETA, S(contig(B_, HV)), state, S(sts or contig(B_, HV, dk, DVN)), o,
                                  S(os_ or contig(B_, HV, DVN)), B_, Hk, HV, dk, DVN, 0.1, 1e-6, dt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(state=P(0)), INVALID), (dict(o=SI), INVALID), (dict(o=Q), INVALID), (dict(state=V), INVALID), (dict(dk=130), UNSUP),
    (dict(dt=3), INVALID), (dict(Hk=3), INVALID), (dict(state=P(SI.value + 2)), UNSUP),
    (dict(sts=[0, DKN * DVN, DVN, 1]), INVALID),  # every sequence the same state
    (dict(sts=[HV * DKN * DVN, DKN * DVN, 1, DKN]), UNSUP), (dict(os_=[HV * DVN, DVN, 2]), UNSUP)])
def test_delta_step_validation(lib, kw, status):
    assert step(lib, **kw) == status


def test_delta_workspace_queries(lib):
    w = lambda f, *a: getattr(lib, f"dynconv_delta_{f}_workspace_size")(*a)  # noqa: E731
    for dt in (F32, BF16, F16):
        f, b = w("fwd", 2, 100, 2, 4, 64, 64, dt), w("bwd", 2, 100, 2, 4, 64, 64, dt)
        assert 0 < f < b
        assert w("fwd", 2, 100, 2, 4, 64, 64, dt) < w("fwd", 2, 200, 2, 4, 64, 64, dt)
    for bad in ((2, 100, 3, 4, 64, 64, BF16), (2, 100, 2, 4, 200, 64, BF16), (2, 100, 2, 4, 64, 64, 5), (2, 0, 2, 4, 64, 64, BF16),
                (0, 100, 2, 4, 64, 64, BF16), (-2, 100, 2, 4, 64, 64, BF16)):
        assert w("fwd", *bad) == 0 and w("bwd", *bad) == 0
    # extreme sizes stay finite and positive (no wrap): 2^31 bytes are passed long before the limits
    assert w("bwd", 1, 2**30, 1, 1, 128, 128, BF16) > 2**40


def nfwd(lib, x=Q, xs=None, w=K, z=None, r=None, after=0, y=O, ys=None, h=None, n=(2, 3, 4), D=40, eps=1e-6, dt=BF16):
    c = contig(*n, D)
    return lib.dynconv_norm_fwd(x, S(xs or c), w, z, S(c) if z else None, r, S(c) if r else None, after, 0.5, y, S(ys or c), h,
                                S(c) if h else None, *n, D, eps, dt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=P(0)), INVALID), (dict(y=P(0)), INVALID), (dict(y=Q), INVALID), (dict(y=K), INVALID), (dict(dt=4), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(n=(2, -3, 4)), INVALID), (dict(D=-1), INVALID),
    (dict(D=(1 << 24) + 1), UNSUP), (dict(n=(2**20, 2**11, 1)), UNSUP), (dict(n=(2**40, 1, 1)), UNSUP),
    (dict(r=V), INVALID),                  # a residual before the norm needs h
    (dict(r=V, h=V), INVALID), (dict(r=V, h=O), INVALID), (dict(z=V, y=V), INVALID),
    (dict(xs=[480, 160, 40, 2]), UNSUP), (dict(xs=[480, -160, 40, 1]), UNSUP), (dict(x=P(Q.value + 1)), UNSUP),
    (dict(w=P(K.value + 1)), UNSUP), (dict(ys=[480, 0, 40, 1]), INVALID),
    (dict(n=(0, 3, 4)), OK), (dict(D=0), OK)])
def test_norm_fwd_validation(lib, kw, status):
    assert nfwd(lib, **kw) == status


def nbwd(lib, x=Q, w=K, z=None, dz=None, dy=DO, dh=None, at=0, dx=DQ, dres=None, dw=DG, ws=None, wsb=0, n=(2, 3, 4), D=40,
         eps=1e-6):
    c = contig(*n, D)
    t = lambda p: (p, S(c) if p else None)  # noqa: E731
    return lib.dynconv_norm_bwd(*t(x), w, *t(z), *t(dy), *t(dh), at, 0.5, *t(dx), *t(dres), dw, *t(dz), *n, D, eps, BF16, ws, wsb,
                                None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=P(0)), INVALID), (dict(dy=P(0)), INVALID), (dict(dx=P(0)), INVALID), (dict(dx=DO), INVALID), (dict(dx=Q), INVALID),
    (dict(at=3), INVALID), (dict(at=-1), INVALID), (dict(at=0, dh=V), INVALID), (dict(at=2, dres=V), INVALID),
    (dict(z=V), INVALID),                  # a gate's gradient needs a place
    (dict(dz=V), INVALID), (dict(z=V, dz=DQ), INVALID), (dict(at=1, dres=DQ), INVALID), (dict(dw=P(DQ.value)), INVALID),
    (dict(dw=P(DG.value + 2)), UNSUP), (dict(eps=-1.0), INVALID), (dict(), WORKSPACE), (dict(ws=WS, wsb=8), WORKSPACE),
    (dict(D=0), OK), (dict(n=(0, 1, 1), dw=None), OK)])
def test_norm_bwd_validation(lib, kw, status):
    assert nbwd(lib, **kw) == status


def test_norm_workspace_query(lib):
    f = lib.dynconv_norm_bwd_workspace_size
    assert f(1, 1, 5, 64, BF16) >= 64 * 4 and f(0, 1, 5, 64, BF16) == 0 and f(1, 1, 5, 64, 7) == 0
    assert f(1, 1, 10**6, 64, BF16) <= 1024 * 64 * 4


# ---------------------------------------------------------------------------------
# Bindings
# ---------------------------------------------------------------------------------


def tens(T=6, Hk=2, Hv=4, dk=8, dv=16, dtype=torch.bfloat16):
    return (torch.zeros(1, T, Hk, dk, dtype=dtype), torch.zeros(1, T, Hk, dk, dtype=dtype),
            torch.zeros(1, T, Hv, dv, dtype=dtype), torch.zeros(1, T, Hv), torch.zeros(1, T, Hv, dtype=dtype))


def test_delta_binding_checks():
    q, k, v, g, b = tens()
    do = torch.zeros_like(v)
    with pytest.raises(RuntimeError, match="GPU only"):
        dc.dynconv_delta_fwd(q, k, v, g, b)
    with pytest.raises(RuntimeError, match="GPU only"):
        dc.dynconv_delta_bwd(q, k, v, g, b, do)
    for bad in ((q[0], k, v, g, b), (q, k, v[0], g, b), (q, k[:, :5], v, g, b), (q, k, v, g[:, :5], b), (q, k, v, g, b[..., :3]),
                (q[:, :, :0], k[:, :, :0], v, g, b), (q.expand(1, 6, 2, 8), k, v[:, :, :3], g[..., :3], b[..., :3])):
        with pytest.raises(ValueError):
            dc.dynconv_delta_fwd(*bad)
    for bad in ((q, k, v, g.bfloat16(), b), (q, k, v, g, b.float()), (q.float(), k, v, g, b), (q.double(), k.double(), v, g, b)):
        with pytest.raises(TypeError):
            dc.dynconv_delta_fwd(*bad)
    with pytest.raises(ValueError, match="qk_norm_eps"):
        dc.dynconv_delta_fwd(q, k, v, g, b, qk_norm_eps=-1.0)
    with pytest.raises(ValueError, match="state"):
        dc.dynconv_delta_fwd(q, k, v, g, b, state=torch.zeros(1, 4, 8, 15))
    with pytest.raises(TypeError, match="state"):
        dc.dynconv_delta_fwd(q, k, v, g, b, state=torch.zeros(1, 4, 8, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="do"):
        dc.dynconv_delta_bwd(q, k, v, g, b, do[:, :3])
    with pytest.raises(ValueError, match="out"):
        dc.dynconv_delta_fwd(q, k, v, g, b, out=torch.zeros(1, 6, 4, 15, dtype=torch.bfloat16))
    one = [t[:, 0] for t in (q, k, v, g, b)]
    with pytest.raises(ValueError, match="state"):
        dc.dynconv_delta_step(*one, None)
    with pytest.raises(RuntimeError, match="GPU only"):
        dc.dynconv_delta_step(*one, torch.zeros(1, 4, 8, 16))
    with pytest.raises(ValueError):
        dc.dynconv_delta_step(q, k, v, g, b, torch.zeros(1, 4, 8, 16))


@pytest.mark.parametrize("Hk,Hv,dk,dv", [(1, 1, 0, 8), (1, 1, 8, 0), (1, 0, 8, 8), (0, 0, 8, 8)])
def test_delta_binding_refuses_empty_heads(Hk, Hv, dk, dv):
    """They would leave outputs of the other sizes unwritten."""
    q, v, g = torch.zeros(1, 3, Hk, dk), torch.zeros(1, 3, Hv, dv), torch.zeros(1, 3, Hv)
    with pytest.raises(ValueError, match="heads"):
        dc.dynconv_delta_fwd(q, q, v, g, g)
    with pytest.raises(ValueError, match="heads"):
        dc.dynconv_delta_bwd(q, q, v, g, g, v)


def test_norm_binding_checks():
    x, w = torch.zeros(2, 3, 8), torch.ones(8)
    for kw in (dict(gate=x[:1]), dict(residual=x[..., :4]), dict(out=x[0]), dict(residual_at="inside"), dict(out_h=x)):
        with pytest.raises(ValueError):
            dc.dynconv_norm_fwd(x, w, **kw)
    for bad in (torch.ones(7), torch.ones(16)[::2]):
        with pytest.raises(ValueError):
            dc.dynconv_norm_fwd(x, bad)
    with pytest.raises(TypeError):
        dc.dynconv_norm_fwd(x, w.half())
    with pytest.raises(ValueError):
        dc.dynconv_norm_fwd(torch.zeros(1, 1, 1, 1, 8))
    with pytest.raises(ValueError):
        dc.dynconv_norm_fwd(torch.zeros(()))
    for kw in (dict(dh=x), dict(residual_at="inside"), dict(dh=x, residual_at="after")):
        with pytest.raises(ValueError):
            dc.dynconv_norm_bwd(x, w, x, **kw)
    with pytest.raises(RuntimeError, match="GPU only"):
        dc.dynconv_norm_fwd(x, w)


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
