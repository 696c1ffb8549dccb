"""GPU parity of the gated linear scan and of activations in 8 bits against the float64 oracle, through
the bindings.

Tolerances: element by element the running error bound of tests/scan_bounds.py, and half a step of the
stored type (2^-8 of the value in bfloat16, 2^-11 in float16 and, below its smallest normal value, 2^-25).
"""
import numpy as np
import pytest
import torch

import dynamic_short_convolution_amd as dc
import synth
from dynamic_short_convolution_amd import DynconvError
from oracle import held8, pack8, scan_bwd, scan_fwd
from tests.parity import to64
from tests.scan_bounds import bwd_bounds, fwd_bound

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
TINY = {torch.float32: 2.0**-126, torch.bfloat16: 2.0**-126, torch.float16: 2.0**-25}


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    yield
    torch.cuda.synchronize()


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    return (torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)) * scale).to(dtype).cuda()


def rates(seed, D):
    return torch.from_numpy(-8.0 * np.log(0.9 + 0.099 * np.random.default_rng(seed).random(D))).float().cuda()


def near(name, got, ref, bound):
    """|got - ref| <= bound + half a step of got's type."""
    g, ref = to64(got), np.asarray(ref, dtype=np.float64)
    assert g.shape == ref.shape, f"{name}: {g.shape} != {ref.shape}"
    off = np.abs(g - ref) - (bound + HALF[got.dtype] * (np.abs(ref) + bound) + TINY[got.dtype])
    if off.size and not (off <= 0).all():
        i = np.unravel_index(np.argmax(np.where(np.isnan(off), np.inf, off)), off.shape)
        raise AssertionError(f"{name} at {i}: got {g[i]!r} ref {ref[i]!r} bound {np.broadcast_to(bound, ref.shape)[i]!r}; "
                             f"{int((~(off <= 0)).sum())} of {off.size}")


def opt(t):
    return None if t is None else to64(t)


def inputs(B, T, D, dtype, gated=True, docs=0, state=True, seed=1):
    td = TD[dtype]
    s = {"x": rand(seed, B, T, D, dtype=td), "decay": rand(seed + 1, B, T, D, dtype=td), "rate": rates(seed + 2, D)}
    s["gate"] = rand(seed + 3, B, T, D, dtype=td) if gated else None
    s["seq_idx"] = synth.segments(B, T, docs, seed, first=(1, 2)).cuda() if docs else None
    s["state"] = rand(seed + 4, B, D) if state else None
    return s, rand(seed + 5, B, T, D, dtype=td), rand(seed + 6, B, D)


def check(s, dy, dlast):
    x, decay, rate, gate, seq, state = (opt(s[n]) for n in ("x", "decay", "rate", "gate", "seq_idx", "state"))
    seq = None if seq is None else seq.astype(np.int64)
    args = (x, decay, rate, gate)
    y, last, chunks = dc.dynconv_scan_fwd(**s, want_state=True, want_chunks=True)
    ry, rlast = scan_fwd(*args, seq, state)
    bound = fwd_bound(*args, seq, state)
    near("y", y, ry, bound)
    near("state", last, rlast, bound[:, -1])
    starts = np.concatenate([np.zeros_like(rlast)[:, None] if state is None else state[:, None], ry[:, 127:-1:128]], 1)
    near("chunks", chunks, starts, np.concatenate([np.zeros_like(rlast)[:, None], bound[:, 127:-1:128]], 1))
    ref = scan_bwd(*args, to64(dy), seq, state, opt(dlast))
    bounds = bwd_bounds(*args, to64(dy), seq, state, opt(dlast))
    for kept in (chunks, None):
        got = dc.dynconv_scan_bwd(**s, dy=dy, chunks=kept, dstate_out=dlast, need_dstate=True)
        for name, g, r, b in zip(("dx", "ddecay", "drate", "dgate", "dstate"), got, ref, bounds):
            assert (g is None) == (r is None)
            if g is not None:
                near(f"{name}, {'kept' if kept is not None else 'recomputed'} states", g, r, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gated,docs,state", [(True, 0, True), (False, 7, False), (True, 40, True)])
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 5, 2), (1, 64, 63), (2, 127, 64), (1, 128, 65), (3, 129, 70), (1, 255, 130),
                                   (1, 256, 66), (2, 257, 96), (1, 700, 33)], ids=str)
def test_against_oracle(shape, gated, docs, state, dtype):
    check(*inputs(*shape, dtype, gated, docs, state))


@pytest.mark.parametrize("dtype,shape,docs", [("bf16", (1, 4097, 64), 0), ("f32", (1, 5000, 65), 300), ("f16", (2, 3000, 130), 0),
                                              ("f32", (1, 9000, 2), 2000)], ids=str)
def test_segments_of_long_sequences(dtype, shape, docs):
    """Few channels: the sequence is cut into segments that run at the same time."""
    assert dc._lib.load().dynconv_scan_fwd_workspace_size(*shape, 0) > 0
    check(*inputs(*shape, dtype, True, docs, True, seed=20))


@pytest.mark.parametrize("dtype,docs", [("bf16", 0), ("f32", 20)])
@pytest.mark.parametrize("shape", [(128, 515, 3), (16, 641, 500)], ids=str)
def test_only_the_backward_is_cut(shape, dtype, docs):
    """128 workgroups: the forward, which the backward may repeat, runs whole."""
    assert dc._lib.load().dynconv_scan_fwd_workspace_size(*shape, 0) == 0
    B, T, D = shape
    one = dc._lib.load().dynconv_scan_bwd_workspace_size(B, T, D, 1, 0)
    assert one >= 2 * B * D * 4 + 2 * B * D * 8  # two segments' partial sums and maps
    check(*inputs(*shape, dtype, True, docs, True, seed=25))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("docs", [0, 9])
@pytest.mark.parametrize("shape", [(1, 1, 3), (2, 130, 64), (1, 300, 129), (2, 257, 200), (1, 2100, 66)], ids=str)
def test_backward_of_packed_inputs(shape, docs, dtype):
    """The gradients at the values that the codes stand for."""
    s, dy, dlast = inputs(*shape, dtype, True, docs, True, seed=40)
    packed = {n: dc.dynconv_pack8(s[n]) for n in ("x", "decay", "gate")}
    held = [held8(to64(s[n])) for n in ("x", "decay", "gate")]
    seq = None if s["seq_idx"] is None else s["seq_idx"].cpu().numpy()
    rest = (to64(dy), seq, to64(s["state"]), to64(dlast))
    args = (held[0], held[1], to64(s["rate"]), held[2])
    ref, bounds = scan_bwd(*args, *rest), bwd_bounds(*args, *rest)
    got = dc.dynconv_scan_bwd(**{**s, **packed}, dy=dy, dstate_out=dlast, need_dstate=True)
    for name, g, r, b in zip(("dx", "ddecay", "drate", "dgate", "dstate"), got, ref, bounds):
        near(name, g, r, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,D,gated", [(1, 1, True), (3, 64, False), (5, 515, True), (2, 2048, True)])
def test_steps_continue_the_scan(B, D, gated, dtype):
    s, _, _ = inputs(B, 6, D, dtype, gated, 0, True, seed=60)
    args = tuple(opt(s[n]) for n in ("x", "decay", "rate", "gate"))
    ry, rlast = scan_fwd(*args, None, to64(s["state"]))
    bound = fwd_bound(*args, None, to64(s["state"]))
    state = s["state"].clone()
    for t in range(6):
        y = dc.dynconv_scan_step(s["x"][:, t], s["decay"][:, t], s["rate"], state, gate=None if s["gate"] is None else s["gate"][:, t])
        near(f"token {t}", y, ry[:, t], bound[:, t])
    near("state", state, rlast, bound[:, -1])


def test_gradients_are_differences():
    """Central differences of the kernels' own forward in float32, summed in 64 bits. Allowed: what the
    oracle's difference of the same step is off from its gradient, and the forward's error bound over the step."""
    s, dy, dlast = inputs(1, 40, 3, "f32", True, 11, True, seed=80)
    got = dc.dynconv_scan_bwd(**s, dy=dy, dstate_out=dlast, need_dstate=True)
    grads = dict(zip(("x", "decay", "rate", "gate", "state"), got))
    s64 = {n: to64(t) for n, t in s.items()}
    names = ("x", "decay", "rate", "gate", "seq_idx", "state")
    exact = dict(zip(("x", "decay", "rate", "gate", "state"),
                     scan_bwd(*(s64[n] for n in names[:4]), to64(dy), s64["seq_idx"], s64["state"], to64(dlast))))
    bound = fwd_bound(*(s64[n] for n in names))
    h = 2.0**-5
    noise = 1.5 * ((np.abs(to64(dy)) * bound).sum() + (np.abs(to64(dlast)) * bound[:, -1]).sum()) / h

    def loss():
        y, last = dc.dynconv_scan_fwd(**s, want_state=True)
        return float((y.double() * dy.double()).sum() + (last.double() * dlast.double()).sum())

    def loss64():
        y, last = scan_fwd(*(s64[n] for n in names))
        return float((y * to64(dy)).sum() + (last * to64(dlast)).sum())

    def difference(t, at, value):
        keep = float(t[at])
        t[at] = np.float32(keep + h).item()
        up, hi = value(), float(t[at])
        t[at] = np.float32(keep - h).item()
        down, lo = value(), float(t[at])
        t[at] = keep
        return (up - down) / (hi - lo)

    for name, at in (("x", (0, 17, 1)), ("decay", (0, 3, 2)), ("decay", (0, 30, 0)), ("rate", (1,)), ("gate", (0, 39, 2)), ("state", (0, 0))):
        off = abs(difference(s64[name], at, loss64) - exact[name][at])
        assert off < 0.1 * max(1.0, abs(exact[name][at])) and noise < 0.05  # both small beside gradients of order 1
        assert abs(difference(s[name], at, loss) - float(grads[name][at])) <= 1.01 * off + noise, (name, at)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_extreme_gates(dtype):
    """Closed decay gates (a = 1, nothing taken in), open ones with large rates (a = 0), closed and open input gates."""
    s, dy, dlast = inputs(1, 300, 8, dtype, True, 0, True, seed=90)
    big = 60.0
    s["decay"][:, :, 0], s["decay"][:, :, 1] = -big, big
    s["gate"][:, :, 2], s["gate"][:, :, 3] = -big, big
    s["rate"][4:6] = 0.0
    s["rate"][1], s["rate"][6] = 1e4, 200.0
    y, last, chunks = dc.dynconv_scan_fwd(**s, want_state=True, want_chunks=True)
    for g in (y, last, chunks):
        assert bool(torch.isfinite(g).all())
    # a rate of zero: the state passes unchanged, bit for bit
    assert torch.equal(last[:, 4:6], s["state"][:, 4:6])
    # a of zero: every token stands alone, b = 1
    alone = torch.sigmoid(s["gate"][:, :, 1].double()) * s["x"][:, :, 1].double()
    near("alone", y[:, :, 1], to64(alone), 40 * 2.0**-24 * np.abs(to64(alone)))
    got = dc.dynconv_scan_bwd(**s, dy=dy, chunks=chunks, dstate_out=dlast, need_dstate=True)
    for g in got:
        assert bool(torch.isfinite(g).all())
    assert float(got[1][:, :, 4:6].abs().max()) == 0.0 and float(got[0][:, :, 4:6].abs().max()) == 0.0
    near("dstate of an unchanged state", got[4][:, 4], to64(dy.double()[:, :, 4].sum(1) + dlast.double()[:, 4]),
         40 * 300 * 2.0**-24 * to64(dy.double()[:, :, 4].abs().sum(1) + 1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_stays_in_its_channel_and_document(dtype, bad):
    s, dy, _ = inputs(1, 600, 70, dtype, True, 0, False, seed=100)
    seq = torch.zeros(1, 600, dtype=torch.int32)
    seq[:, 150:], seq[:, 411:] = 1, 2
    s["seq_idx"] = seq.cuda()
    clean = dc.dynconv_scan_fwd(**s, want_state=True)
    cg = dc.dynconv_scan_bwd(**s, dy=dy)
    for name in ("x", "decay", "gate"):
        keep = s[name][0, 200, 5].clone()
        s[name][0, 200, 5] = float("nan") if name != "x" else bad
        y, last = dc.dynconv_scan_fwd(**s, want_state=True)
        assert bool((~torch.isfinite(y[0, 200:411, 5])).any())
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[0, 150:411, 5] = True
        assert torch.equal(y[~hit], clean[0][~hit]) and torch.equal(last, clean[1])
        assert torch.equal(y[0, 150:200, 5], clean[0][0, 150:200, 5])
        for g, c in zip(dc.dynconv_scan_bwd(**s, dy=dy), cg):
            if g is None:
                continue
            if g.dim() == 3:
                assert torch.equal(g[~hit], c[~hit]), name
            else:
                keep_ch = torch.arange(70) != 5
                assert torch.equal(g[keep_ch], c[keep_ch])
        s[name][0, 200, 5] = keep


@pytest.mark.parametrize("docs", [0, 3])
@pytest.mark.parametrize("T", [5, 128, 200])
def test_infinity_in_the_last_token(T, docs):
    """dl of that token is the infinity dh sigmoid(gate) x a^2 / b, the others are finite: drate is infinite, with
    a tile's rows behind the last token and without."""
    s, _, _ = inputs(2, T, 3, "f32", True, docs, True, seed=45)
    s["x"][1, T - 1, 1] = float("inf")
    dx, ddecay, drate, dgate, dstate = dc.dynconv_scan_bwd(**s, dy=torch.ones(2, T, 3, device="cuda"), need_dstate=True)
    assert drate[1].item() == float("inf") and torch.isfinite(drate[[0, 2]]).all()
    for t in (ddecay, dgate):
        assert t[1, T - 1, 1].isinf()
        t[1, T - 1, 1] = 0.0
        assert torch.isfinite(t).all()
    assert torch.isfinite(dx).all() and torch.isfinite(dstate).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 63), ("f32", 130), ("f16", 100)])
def test_strided_views_inside_guard_bands(dtype, D):
    td = TD[dtype]
    B, T = 2, 300
    s, dy, _ = inputs(B, T, D, dtype, True, 20, True, seed=110)

    def inside(t, off, fill=float("nan")):
        big = torch.full((T + 1, B + 1, D + 7 + off), fill, dtype=td, device="cuda")
        v = big[:-1, 1:, off:off + D].permute(1, 0, 2)
        v.copy_(t)
        return big, v

    ref = dc.dynconv_scan_fwd(**s, want_state=True, want_chunks=True)
    args, rest = tuple(to64(s[n]) for n in ("x", "decay", "rate", "gate")), (s["seq_idx"].cpu().numpy(), to64(s["state"]))
    (ry, rlast), bound = scan_fwd(*args, *rest), fwd_bound(*args, *rest)
    rg, bounds = scan_bwd(*args, to64(dy), *rest), bwd_bounds(*args, to64(dy), *rest)
    for off in (0, 1):
        v = dict(s)
        for n in ("x", "decay", "gate"):
            v[n] = inside(s[n], off)[1]
        big, out = inside(torch.zeros(B, T, D, dtype=td, device="cuda"), off)
        # one channel per lane where the rows' strides are odd: runs of other lengths, so other roundings
        y, last, chunks = dc.dynconv_scan_fwd(**v, want_state=True, want_chunks=True, out=out)
        near("y", y, ry, bound)
        near("state", last, rlast, bound[:, -1])
        assert int(torch.isfinite(big).sum()) == B * T * D
        for name, g, r, b in zip(("dx", "ddecay", "drate", "dgate"), dc.dynconv_scan_bwd(**v, dy=inside(dy, off)[1], chunks=chunks),
                                 rg, bounds):
            near(name, g, r, b)
    # ids and states of other layouts
    v = dict(s, seq_idx=s["seq_idx"].t().contiguous().t(), state=torch.cat([s["state"], s["state"]], 1)[:, :D])
    assert all(torch.equal(a, b) for a, b in zip(dc.dynconv_scan_fwd(**v, want_state=True, want_chunks=True), ref))


def test_broadcast_inputs():
    s, dy, _ = inputs(3, 140, 64, "bf16", True, 0, True, seed=120)
    for n in ("x", "decay", "gate"):
        s[n] = s[n][:1, :1].expand(3, 140, 64)
    c = {n: t.contiguous() if torch.is_tensor(t) else t for n, t in s.items()}
    assert torch.equal(dc.dynconv_scan_fwd(**s), dc.dynconv_scan_fwd(**c))
    for a, b in zip(dc.dynconv_scan_bwd(**s, dy=dy[:1].expand(3, 140, 64)), dc.dynconv_scan_bwd(**c, dy=dy[:1].repeat(3, 1, 1))):
        assert (a is None and b is None) or torch.equal(a, b)


def test_one_token_of_any_stride():
    s, dy, dlast = inputs(2, 1, 64, "bf16", True, 0, True, seed=125)
    v = dict(s)
    for n in ("x", "decay", "gate"):
        big = torch.full((2, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        big[:, 1] = s[n][:, 0]
        v[n] = big.as_strided((2, 1, 64), (128, 1 << 30, 1), 64)
    assert torch.equal(dc.dynconv_scan_fwd(**v), dc.dynconv_scan_fwd(**s))
    for a, b in zip(dc.dynconv_scan_bwd(**v, dy=dy), dc.dynconv_scan_bwd(**s, dy=dy)):
        assert (a is None and b is None) or torch.equal(a, b)


def test_a_single_token_of_the_widest_rows():
    """2^24 channels of float32: both directions at the first, the last and some channels between."""
    D = 2**24
    g = torch.Generator(device="cuda").manual_seed(15)
    x, decay, dy = (torch.randn(1, 1, D, device="cuda", generator=g) for _ in range(3))
    rate, state = torch.rand(D, device="cuda", generator=g), torch.randn(1, D, device="cuda", generator=g)
    at = np.r_[0:64, 2**20 - 3:2**20 + 3, D - 64:D]
    part = [to64(t[..., at]) for t in (x, decay, rate, dy, state)]
    px, pd, pr, pdy, ps = part
    near("y", dc.dynconv_scan_fwd(x, decay, rate, state=state)[..., at], scan_fwd(px, pd, pr, state=ps)[0],
         fwd_bound(px, pd, pr, state=ps))
    got = dc.dynconv_scan_bwd(x, decay, rate, dy, state=state, need_dstate=True)
    ref, bounds = scan_bwd(px, pd, pr, None, pdy, state=ps), bwd_bounds(px, pd, pr, None, pdy, state=ps)
    for name, t, r, b in zip(("dx", "ddecay", "drate", "dgate", "dstate"), got, ref, bounds):
        if t is not None:
            near(name, t[..., at], r, b)


def test_offsets_past_32_bits():
    s, dy, _ = inputs(2, 130, 64, "bf16", True, 0, False, seed=130)
    far = torch.zeros(2**31 + 130 * 64, dtype=torch.bfloat16, device="cuda").as_strided((2, 130, 64), (2**31, 64, 1))
    far.copy_(s["x"])
    out = torch.zeros(2**31 + 130 * 64, dtype=torch.bfloat16, device="cuda").as_strided((2, 130, 64), (2**31, 64, 1))
    ref = dc.dynconv_scan_fwd(**s)
    assert torch.equal(dc.dynconv_scan_fwd(**dict(s, x=far), out=out), ref)
    # rows 2^22 - 2 elements apart: a tile's 256 rows span 2^31 bytes
    wide = torch.zeros(257 * (2**22 - 2) + 64, dtype=torch.bfloat16, device="cuda").as_strided((1, 257, 64), (2**30, 2**22 - 2, 1))
    t, dt, _ = inputs(1, 257, 64, "bf16", True, 0, False, seed=131)
    wide.copy_(t["x"])
    w = dict(t, x=wide)
    assert torch.equal(dc.dynconv_scan_fwd(**w), dc.dynconv_scan_fwd(**t))
    for a, b in zip(dc.dynconv_scan_bwd(**w, dy=dt), dc.dynconv_scan_bwd(**t, dy=dt)):
        assert (a is None and b is None) or torch.equal(a, b)


def test_states_in_place_and_empty():
    s, dy, dlast = inputs(2, 1100, 64, "bf16", True, 0, True, seed=140)
    y, last = dc.dynconv_scan_fwd(**s, want_state=True)
    st = s["state"].clone()
    y2, l2 = dc.dynconv_scan_fwd(**dict(s, state=st), state_out=st)
    assert l2 is st and torch.equal(st, last) and torch.equal(y, y2)
    # two halves are the whole up to the rounding of the order of sums
    a = {n: t[:, :600] if n in ("x", "decay", "gate") else t for n, t in s.items()}
    b = {n: t[:, 600:] if n in ("x", "decay", "gate") else t for n, t in s.items()}
    _, mid = dc.dynconv_scan_fwd(**a, want_state=True)
    _, end = dc.dynconv_scan_fwd(**dict(b, state=mid), want_state=True)
    args = tuple(opt(s[n]) for n in ("x", "decay", "rate", "gate"))
    bound = fwd_bound(*args, None, to64(s["state"]))[:, -1]
    assert (np.abs(to64(end) - to64(last)) <= 2 * bound).all()
    empty = {n: t[:, :0] if n in ("x", "decay", "gate") else t for n, t in s.items()}
    y, last, chunks = dc.dynconv_scan_fwd(**empty, want_state=True, want_chunks=True)
    assert y.shape == (2, 0, 64) and torch.equal(last, s["state"]) and chunks.shape == (2, 0, 64)
    got = dc.dynconv_scan_bwd(**empty, dy=dy[:, :0], dstate_out=dlast, need_dstate=True)
    assert torch.equal(got[4], dlast) and float(got[2].abs().max()) == 0.0
    got = dc.dynconv_scan_bwd(**empty, dy=dy[:, :0], need_dstate=True)
    assert float(got[4].abs().max()) == 0.0
    none = {n: t[:0] if n in ("x", "decay", "gate", "state") else t for n, t in s.items()}
    assert dc.dynconv_scan_fwd(**none).shape == (0, 1100, 64)
    assert float(dc.dynconv_scan_bwd(**none, dy=dy[:0])[2].abs().max()) == 0.0


def test_same_bits_every_time_captured_and_on_other_streams():
    s, dy, _ = inputs(1, 3000, 192, "bf16", True, 100, True, seed=150)

    def work():
        y, last, chunks = dc.dynconv_scan_fwd(**s, want_state=True, want_chunks=True)
        g = dc.dynconv_scan_bwd(**s, dy=dy, chunks=chunks, need_dstate=True)
        p = {n: dc.dynconv_pack8(s[n]) for n in ("x", "decay", "gate")}
        return [y, last, *g, *dc.dynconv_scan_bwd(**{**s, **p}, dy=dy, need_dstate=True), dc.dynconv_unpack8(p["x"])]

    first = work()
    assert all(torch.equal(a, b) for a, b in zip(first, work()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(4):
        s["x"].copy_(rand(160 + i, 1, 3000, 192))
        s["state"].copy_(rand(170 + i, 1, 192))
        eager = work()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        other = work()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, eager))


# ---------------------------------------------------------------------------------
# Activations in 8 bits
# ---------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 64), (5, 65), (2, 3, 128), (7, 130), (2, 2, 3, 200), (4, 1537), (9, 2048)], ids=str)
def test_pack8_is_the_definition_bit_for_bit(shape, dtype):
    td = TD[dtype]
    x = rand(200, *shape, dtype=td) * torch.exp(4 * rand(201, *shape[:-1], 1)).to(td)
    p = dc.dynconv_pack8(x)
    codes, steps = pack8(to64(x))
    assert np.array_equal(to64(p.codes), codes)
    assert np.array_equal(np.exp2(to64(p.scales) - 127.0), steps)
    back = dc.dynconv_unpack8(p, td)
    held = held8(to64(x))
    assert np.array_equal(to64(back), held)
    assert np.array_equal(to64(dc.dynconv_unpack8(p, torch.float32)), held)
    top = np.abs(to64(x))
    pad = np.pad(top, [(0, 0)] * (x.dim() - 1) + [(0, -shape[-1] % 64)])
    most = np.repeat(pad.reshape(*shape[:-1], -1, 64).max(-1), 64, -1)[..., :shape[-1]]
    assert (np.abs(held - to64(x)) <= 2.0**-7 * most).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_pack8_of_extremes(dtype):
    td = TD[dtype]
    info = torch.finfo(td)
    x = torch.zeros(8, 128, dtype=td, device="cuda")
    x[0, 3], x[0, 70] = info.max, -info.max
    x[1, 1], x[1, 80] = info.smallest_normal, -info.smallest_normal
    x[2, 5] = float("nan")
    x[3, 90] = float("-inf")
    x[4, :64] = torch.arange(64, device="cuda") - 31.5  # ties between codes
    x[5, 0], x[5, 1], x[5, 2] = 127.5, 126.5, 0.5
    x[6, 0] = info.tiny / 2 if dtype != "f16" else 2.0**-24
    back = dc.dynconv_unpack8(dc.dynconv_pack8(x), td)
    want = held8(to64(x))
    assert np.array_equal(to64(back), want, equal_nan=True)
    assert bool(back[2, :64].isnan().all()) and float(back[2, 64:].abs().max()) == 0.0
    assert bool(back[3, 64:].isnan().all()) and float(back[3, :64].abs().max()) == 0.0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_pack8_of_every_width(dtype):
    """Rows shorter than a piece, last pieces that reach back (also into another group), and what stands beside the rows.
    Some float16 groups hold an infinity: they read as NaN."""
    td = TD[dtype]
    for D in [*range(1, 140), 191, 193, 257, 515, 1000, 1025, 16385]:
        x = rand(220 + D, 9, D, dtype=td) * torch.exp(4 * rand(221 + D, 9, 1)).to(td)
        codes, held = pack8(to64(x))[0], held8(to64(x))
        for off in (0, 3):
            guard = torch.full((9, D + 16 + off), 77, dtype=torch.int8, device="cuda")
            p = dc.dynconv_pack8(x, out=dc.Packed8(guard[:, off:off + D], torch.zeros(9, -(-D // 64), dtype=torch.uint8, device="cuda")))
            assert np.array_equal(to64(p.codes), codes), (D, off)
            out = torch.full((9, D + 16 + off), 5.0, dtype=td, device="cuda")
            assert np.array_equal(to64(dc.dynconv_unpack8(p, td, out=out[:, off:off + D])), held, equal_nan=True), (D, off)
            guard[:, off:off + D], out[:, off:off + D] = 77, 5.0
            assert bool((guard == 77).all()) and bool((out == 5.0).all()), (D, off)


def test_pack8_views_and_empty():
    x = rand(210, 6, 5, 130, dtype=torch.bfloat16)
    want = dc.dynconv_pack8(x)
    big = torch.full((5, 6, 140), float("nan"), dtype=torch.bfloat16, device="cuda")
    for off in (0, 1):
        v = big[:, :, off:off + 130].permute(1, 0, 2)
        v.copy_(x)
        codes = torch.full((5, 6, 136), 77, dtype=torch.int8, device="cuda")
        out = dc.Packed8(codes[:, :, off:off + 130].permute(1, 0, 2), torch.zeros(6, 5, 4, dtype=torch.uint8, device="cuda")[..., :3])
        got = dc.dynconv_pack8(v, out=out)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
        codes[:, :, off:off + 130] = 77
        assert bool((codes == 77).all())
    wide = rand(211, 40, 256, dtype=torch.float32)
    out = torch.full((40, 260), float("nan"), device="cuda")
    dc.dynconv_unpack8(dc.dynconv_pack8(wide), torch.float32, out=out[:, 4:])
    assert np.array_equal(to64(out[:, 4:]), held8(to64(wide))) and bool(out[:, :4].isnan().all())
    assert dc.dynconv_pack8(x[:0]).codes.shape == (0, 5, 130)
    assert dc.dynconv_unpack8(dc.dynconv_pack8(x[:, :, :0]), torch.float16).shape == (6, 5, 0)


def test_refusals():
    s, dy, _ = inputs(2, 10, 64, "bf16", True, 0, True, seed=220)
    p = dc.dynconv_pack8(s["x"])
    with pytest.raises(DynconvError, match="INVALID_ARG"):
        dc.dynconv_scan_fwd(**s, out=s["x"])
    with pytest.raises(RuntimeError):
        dc.dynconv_scan_fwd(**dict(s, rate=s["rate"].cpu()))
    with pytest.raises(ValueError):
        dc.dynconv_scan_bwd(**dict(s, x=p), dy=dy)
    with pytest.raises(ValueError):
        dc.dynconv_scan_bwd(**dict(s, gate=p), dy=dy)
    with pytest.raises(DynconvError, match="INVALID_ARG"):
        dc.dynconv_scan_step(s["x"][:, 0], s["decay"][:, 0], s["rate"], s["state"], out=s["x"][:, 0])
    with pytest.raises(DynconvError, match="UNSUPPORTED"):
        dc.dynconv_pack8(rand(221, 64, 4).t())


def test_many_short_sequences():
    B, T, D = 70001, 2, 64
    s, dy, _ = inputs(B, T, D, "bf16", True, 0, True, seed=230)
    y, last = dc.dynconv_scan_fwd(**s, want_state=True)
    g = dc.dynconv_scan_bwd(**s, dy=dy, need_dstate=True)
    pick = slice(B - 40, B)
    part = {n: t if n == "rate" or t is None else t[pick] for n, t in s.items()}
    args = tuple(opt(part[n]) for n in ("x", "decay", "rate", "gate"))
    bound = fwd_bound(*args, None, to64(part["state"]))
    ry, rlast = scan_fwd(*args, None, to64(part["state"]))
    near("y", y[pick], ry, bound)
    near("state", last[pick], rlast, bound[:, -1])
    ref, bounds = scan_bwd(*args, to64(dy[pick]), None, to64(part["state"])), bwd_bounds(*args, to64(dy[pick]), None, to64(part["state"]))
    for name, i in (("dx", 0), ("ddecay", 1), ("dgate", 3), ("dstate", 4)):
        near(name, g[i][pick], ref[i], bounds[i])


def test_long_narrow_sequence_of_all_segments():
    s, dy, dlast = inputs(1, 40000, 3, "f32", True, 5000, True, seed=240)
    check(s, dy, dlast)
