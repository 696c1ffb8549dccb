"""GPU parity of the group norm (channels last; per token and over sequences) against the float64 oracle,
through the bindings.

Tolerances: element by element a running error bound (`bounds` below, u = 2^-24), and half a step of the
stored type. A sum over a group goes through at most 32 additions in a lane and 8 between lanes: 40 u
of the sum of magnitudes; with its division 48 u. x - mean is then off by 48 u mean|x| + u |x|, 1 / sqrt(var + eps)
relatively by that over the deviation and 48 u; a sigmoid by (|z| + 5) u of itself; the gradients' sums by 48 u of
their magnitudes, the parameters' by (48 + rows of a lane) u.
"""
import numpy as np
import pytest
import torch

import dynamic_short_convolution_amd as dc
from dynamic_short_convolution_amd import DynconvError
from oracle import groupnorm_bwd, groupnorm_fwd, held8
from oracle.delta_oracle import _silu
from tests.parity import to64

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
TINY = {torch.float32: 2.0**-126, torch.bfloat16: 2.0**-126, torch.float16: 2.0**-25}
U = 2.0**-24


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    yield
    torch.cuda.synchronize()


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    return (torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)) * scale).to(dtype).cuda()


def near(name, got, ref, bound):
    """|got - ref| <= bound + half a step of got's type."""
    g, ref = to64(got), np.asarray(ref, dtype=np.float64)
    assert g.shape == ref.shape, f"{name}: {g.shape} != {ref.shape}"
    off = np.abs(g - ref) - (bound + HALF[got.dtype] * (np.abs(ref) + bound) + TINY[got.dtype])
    if off.size and not (off <= 0).all():
        i = np.unravel_index(np.argmax(np.where(np.isnan(off), np.inf, off)), off.shape)
        raise AssertionError(f"{name} at {i}: got {g[i]!r} ref {ref[i]!r} bound {np.broadcast_to(bound, ref.shape)[i]!r}; "
                             f"{int((~(off <= 0)).sum())} of {off.size}")


def bounds(x, groups, dy, weight=None, bias=None, gate=None, activation=None, over="token", lengths=None, eps=1e-5, rows=64):
    """Bounds of the errors of (y, dx, dweight, dbias, dgate) before any rounding of the result."""
    B, T, C = x.shape
    w = np.ones(C) if weight is None else np.abs(weight)
    out = [np.zeros_like(x) for _ in range(2)] + [np.zeros(C), np.zeros(C), np.zeros_like(x)]
    for b in range(B):
        n = T if lengths is None else int(np.clip(lengths[b], 0, T))
        if n == 0:
            continue

        def mean(t):
            t = t.reshape(n, groups, -1)
            axes = -1 if over == "token" else (0, 2)
            return np.broadcast_to(t.mean(axes, keepdims=True), t.shape).reshape(n, C)

        xb = x[b, :n]
        d = xb - mean(xb)
        rstd = 1.0 / np.sqrt(mean(d * d) + eps)
        norm = d * rstd
        shift = 48 * U * mean(np.abs(xb)) + U * np.abs(xb)
        rel = 48 * U + 2 * mean(shift) * rstd
        dn_ = shift * rstd + rel * np.abs(norm)  # of n
        z = norm * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
        dz_ = w * dn_ + 3 * U * (np.abs(norm) * w + np.abs(0.0 if bias is None else bias))
        sig = (np.abs(z) + 8) * U
        if activation == "silu":
            act, slope = _silu(z)
            act_ = 1.1 * dz_ + sig * np.abs(act)
            slope_ = 0.5 * dz_ + 4 * sig * (1 + np.abs(z))
        else:
            act, slope, act_, slope_ = z, np.ones_like(z), dz_, 0.0
        opened, dopen, open_, dopen_ = 1.0, 0.0, 0.0, 0.0
        if gate is not None:
            g = gate[b, :n]
            opened, dopen = _silu(g)
            open_, dopen_ = (np.abs(g) + 8) * U * np.abs(opened), 4 * (np.abs(g) + 8) * U * (1 + np.abs(g))
        out[0][b, :n] = act_ * np.abs(opened) + np.abs(act) * open_ + 2 * U * np.abs(act * opened)
        up = np.abs(dy[b, :n])
        out[4][b, :n] = up * (act_ * np.abs(dopen) + np.abs(act) * dopen_ + 3 * U * np.abs(act * dopen))
        dz = up * np.abs(opened) * np.abs(slope)
        edz = up * (np.abs(opened) * slope_ + np.abs(slope) * open_) + 4 * U * dz
        out[2] += (edz * np.abs(norm) + dz * dn_ + (48 + rows) * U * dz * np.abs(norm)).sum(0)
        out[3] += (edz + (48 + rows) * U * dz).sum(0)
        # the means over a group: 48 u per token's, the column sums' roundings over a sequence
        terms = (48 + (rows if over == "sequence" else 0)) * U
        e1 = mean(edz * w) + terms * mean(dz * w)
        e2 = mean(edz * w * np.abs(norm) + dz * w * dn_) + terms * mean(dz * w * np.abs(norm))
        m1, m2 = mean(dz * w), mean(dz * w * np.abs(norm))  # of magnitudes: at least the means
        total = dz * w + m1 + np.abs(norm) * m2
        out[1][b, :n] = rstd * (edz * w + e1 + np.abs(norm) * e2 + dn_ * m2 + (6 * U + rel) * total)
    return out


def opt(t):
    return None if t is None else to64(t)


def check(shape, groups, dtype, gated=False, silu=False, over="token", lengths=None, affine=True, seed=1, offset=0.5, packed=False,
          eps=1e-5, rows=64):
    td = TD[dtype]
    C = shape[-1]
    x = (rand(seed, *shape) + offset * rand(seed + 1, C)).to(td)
    dy = rand(seed + 2, *shape, dtype=td)
    kw = dict(weight=(1 + rand(seed + 3, C, scale=0.1)).to(td) if affine else None, bias=rand(seed + 4, C, scale=0.1).to(td) if affine else None,
              gate=rand(seed + 5, *shape, dtype=td) if gated else None, activation="silu" if silu else None, over=over, eps=eps)
    if lengths is not None:
        kw["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    k64 = {n: opt(t) if torch.is_tensor(t) or t is None else t for n, t in kw.items()}
    k64["lengths"] = lengths
    y, stats = dc.dynconv_groupnorm_fwd(x, groups, want_stats=True, **kw)
    x64 = to64(x)
    b = bounds(x64, groups, to64(dy), rows=rows, **k64)
    near("y", y, groupnorm_fwd(x64, groups, **k64), b[0])
    assert (stats is not None) == (over == "sequence")
    xin = x
    if packed:
        xin, x64 = dc.dynconv_pack8(x), held8(x64)
        b = bounds(x64, groups, to64(dy), rows=rows, **k64)
    ref = groupnorm_bwd(x64, groups, to64(dy), **k64)
    for given in ([stats, None] if stats is not None and not packed else [None]):
        dx, dw, db, dg = dc.dynconv_groupnorm_bwd(xin, groups, dy, stats=given, **kw)
        near("dx", dx, ref[0], b[1])
        assert (dw is None) == (db is None) == (not affine)
        if affine:
            near("dweight", dw, ref[1], b[2])
            near("dbias", db, ref[2], b[3])
        assert (dg is None) == (not gated)
        if gated:
            near("dgate", dg, ref[3], b[4])


FORMS = [(False, False), (True, False), (False, True), (True, True)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gated,silu", FORMS)
@pytest.mark.parametrize("shape,groups", [((1, 1, 8), 1), ((2, 5, 64), 4), ((1, 37, 96), 3), ((2, 70, 57), 3), ((1, 9, 171), 3), ((3, 11, 256), 4),
                                          ((1, 13, 520), 4), ((2, 3, 1024), 2), ((1, 5, 2048), 1), ((2, 3, 1500), 2), ((1, 3, 4096), 1),
                                          ((1, 2, 9000), 1), ((1, 3, 2501), 1), ((1, 2, 8192), 1)], ids=str)
def test_per_token(shape, groups, gated, silu, dtype):
    check(shape, groups, dtype, gated, silu)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gated,silu", FORMS)
@pytest.mark.parametrize("shape,groups,lengths", [((1, 1, 16), 2, None), ((2, 5, 64), 4, [5, 2]), ((1, 200, 96), 3, None), ((3, 70, 57), 3, [70, 0, 1]),
                                                  ((2, 300, 171), 3, [299, 300]), ((2, 33, 512), 2, [7, 33]), ((1, 40, 2304), 1, None),
                                                  ((2, 64, 2048), 32, [64, 50]), ((1, 9, 5000), 5, None), ((2, 130, 8), 8, None)], ids=str)
def test_over_sequences(shape, groups, lengths, gated, silu, dtype):
    if shape[-1] == groups:
        pytest.skip("one channel per group") if shape[1] == 1 else None
    check(shape, groups, dtype, gated, silu, over="sequence", lengths=lengths)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("over", ["token", "sequence"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("width,groups", [(1, 5), (2, 64), (3, 9), (4, 16), (5, 7), (7, 64), (8, 32), (9, 300), (11, 3), (15, 5), (16, 64), (17, 3),
                                          (31, 2), (33, 5), (1101, 2), (2049, 1), (4100, 1)])
def test_every_last_piece(width, groups, packed, over, dtype):
    """Groups shorter than a piece of 16 bytes, of some pieces, and with a last one that reaches back into the one before."""
    check((2, 41, width * groups), groups, dtype, True, True, over=over, packed=packed, seed=20,
          lengths=[41, 30] if over == "sequence" else None)


@pytest.mark.parametrize("over", ["token", "sequence"])
def test_elements_of_two_pieces_are_written_the_same(over):
    """Repeated calls give the same bits, those of elements that two lanes write among them."""
    x, dy, gate = (rand(i, 3, 900, 27 * 57, dtype=torch.bfloat16) for i in (21, 22, 23))
    w = rand(24, 27 * 57, dtype=torch.bfloat16)
    kw = dict(weight=w, bias=w, gate=gate, activation="silu", over=over)
    first = (dc.dynconv_groupnorm_fwd(x, 27, **kw), *dc.dynconv_groupnorm_bwd(x, 27, dy, **kw))
    for _ in range(10):
        again = (dc.dynconv_groupnorm_fwd(x, 27, **kw), *dc.dynconv_groupnorm_bwd(x, 27, dy, **kw))
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_sequences(dtype):
    check((2, 5000, 128), 4, dtype, False, True, over="sequence", lengths=[5000, 4097])
    check((40, 2000, 40), 5, dtype, True, False, over="sequence", rows=128)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("over", ["token", "sequence"])
@pytest.mark.parametrize("shape,groups", [((2, 9, 64), 1), ((1, 70, 256), 4), ((2, 33, 130), 2), ((1, 20, 57), 3), ((1, 5, 9000), 1)], ids=str)
def test_backward_of_packed_inputs(shape, groups, over, dtype):
    check(shape, groups, dtype, True, True, over=over, packed=True, seed=30)


@pytest.mark.parametrize("over", ["token", "sequence"])
def test_without_weight_and_bias(over):
    check((2, 20, 96), 4, "bf16", True, True, over=over, affine=False)
    x, w, dy = rand(40, 2, 9, 64), rand(41, 64), rand(42, 2, 9, 64)
    both = dc.dynconv_groupnorm_bwd(x, 4, dy, weight=w, bias=torch.zeros_like(w), over=over)
    one = dc.dynconv_groupnorm_bwd(x, 4, dy, weight=w, over=over)
    assert torch.equal(one[0], both[0]) and torch.equal(one[1], both[1]) and one[2] is None


@pytest.mark.parametrize("tokens,C,groups", [(1, 64, 4), (3, 32, 1), (700, 32, 1), (5000, 64, 2), (2100, 1024, 8), (9, 48, 48 // 16)])
def test_parameter_gradients_over_many_tokens(tokens, C, groups):
    check((1, tokens, C), groups, "f32", True, True, seed=50, rows=64)


@pytest.mark.parametrize("over", ["token", "sequence"])
def test_far_mean_and_constant_rows(over):
    """A mean of 1000 deviations, which the bound of x - mean covers, and groups without any deviation."""
    x = rand(60, 2, 50, 64) + 1000.0
    w, dy = rand(61, 64), rand(62, 2, 50, 64)
    kw = dict(weight=w, over=over)
    k64 = dict(weight=to64(w), over=over)
    y = dc.dynconv_groupnorm_fwd(x, 4, **kw)
    b = bounds(to64(x), 4, to64(dy), **k64)
    near("y", y, groupnorm_fwd(to64(x), 4, **k64), b[0])
    near("dx", dc.dynconv_groupnorm_bwd(x, 4, dy, **kw)[0], groupnorm_bwd(to64(x), 4, to64(dy), **k64)[0], b[1])
    c = torch.full((2, 5, 64), 3.0, device="cuda")
    assert float(dc.dynconv_groupnorm_fwd(c, 4, over=over).abs().max()) == 0.0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_stays_in_its_group(dtype):
    td = TD[dtype]
    x, dy = rand(70, 2, 40, 128, dtype=td), rand(71, 2, 40, 128, dtype=td)
    for over in ("token", "sequence"):
        clean, cg = dc.dynconv_groupnorm_fwd(x, 4, over=over), dc.dynconv_groupnorm_bwd(x, 4, dy, over=over)[0]
        for bad in (float("nan"), float("inf")):
            v = x.clone()
            v[1, 7, 40] = bad
            hit = torch.zeros(2, 40, 128, dtype=torch.bool, device="cuda")
            hit[1, 7 if over == "token" else slice(None), 32:64] = True
            y, g = dc.dynconv_groupnorm_fwd(v, 4, over=over), dc.dynconv_groupnorm_bwd(v, 4, dy, over=over)[0]
            assert torch.equal(y[~hit], clean[~hit]) and torch.equal(g[~hit], cg[~hit])
            assert not bool(torch.isfinite(y[hit]).all()) and not bool(torch.isfinite(g[hit]).all())


def test_tokens_behind_a_sequence():
    """They may hold anything; y, dx and dgate are zero there, and a sequence without tokens has only such."""
    x, gate, dy = rand(80, 3, 70, 64), rand(81, 3, 70, 64), rand(82, 3, 70, 64)
    w = rand(83, 64)
    lengths = torch.tensor([70, 0, 33], dtype=torch.int32, device="cuda")
    kw = dict(weight=w, bias=w, over="sequence", lengths=lengths, activation="silu")
    y, stats = dc.dynconv_groupnorm_fwd(x, 2, gate=gate, want_stats=True, **kw)
    ref = dc.dynconv_groupnorm_bwd(x, 2, dy, gate=gate, stats=stats, **kw)
    for t in (x, gate, dy):
        t[1], t[2, 33:] = float("nan"), float("inf")
    y2, stats2 = dc.dynconv_groupnorm_fwd(x, 2, gate=gate, want_stats=True, **kw)
    got = dc.dynconv_groupnorm_bwd(x, 2, dy, gate=gate, stats=stats2, **kw)
    assert torch.equal(y, y2) and torch.equal(stats, stats2) and all(torch.equal(a, b) for a, b in zip(ref, got))
    for t in (y2, got[0], got[3]):
        assert float(t[1].abs().max()) == 0.0 and float(t[2, 33:].abs().max()) == 0.0
    # lengths outside 0..T are cut to it
    wild = torch.tensor([1000, -5, 33], dtype=torch.int32, device="cuda")
    assert torch.equal(dc.dynconv_groupnorm_fwd(x, 2, gate=gate, **dict(kw, lengths=wild)), y)


def test_two_dimensions_are_tokens():
    x, dy, w = rand(90, 30, 96), rand(91, 30, 96), rand(92, 96)
    assert torch.equal(dc.dynconv_groupnorm_fwd(x, 3, w), dc.dynconv_groupnorm_fwd(x[None], 3, w)[0])
    a, b = dc.dynconv_groupnorm_bwd(x, 3, dy, w), dc.dynconv_groupnorm_bwd(x[None], 3, dy[None], w)
    assert torch.equal(a[0], b[0][0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("over", ["token", "sequence"])
@pytest.mark.parametrize("dtype,C,groups", [("bf16", 128, 2), ("bf16", 66, 2), ("f32", 64, 4), ("f16", 200, 5)])
def test_strided_views_inside_guard_bands(dtype, C, groups, over):
    td = TD[dtype]
    shape = (3, 37, C)

    def inside(t, off):
        big = torch.full((shape[1] + 1, shape[0] + 1, C + 16 + off), float("nan"), dtype=td, device="cuda")
        v = big[:-1, 1:, off:off + C].permute(1, 0, 2)
        v.copy_(t)
        return big, v

    x, gate, dy = (rand(100 + i, *shape, dtype=td) for i in range(3))
    w = rand(103, C, dtype=td)
    k64 = dict(weight=to64(w), gate=to64(gate), over=over)
    ry, rg, b = groupnorm_fwd(to64(x), groups, **k64), groupnorm_bwd(to64(x), groups, to64(dy), **k64), bounds(to64(x), groups, to64(dy), **k64)
    for off in (0, 1):
        (_, xv), (_, gv), (_, dv) = inside(x, off), inside(gate, off), inside(dy, off)
        big, out = inside(torch.zeros(shape, dtype=td, device="cuda"), off)
        dc.dynconv_groupnorm_fwd(xv, groups, weight=w, gate=gv, over=over, out=out)
        near("y", out, ry, b[0])
        assert int(torch.isfinite(big).sum()) == x.numel()
        dx, dw, _, dg = dc.dynconv_groupnorm_bwd(xv, groups, dv, weight=w, gate=gv, over=over)
        near("dx", dx, rg[0], b[1])
        near("dweight", dw, rg[1], b[2])
        near("dgate", dg, rg[3], b[4])


def test_offsets_past_32_bits():
    x = rand(110, 2, 2, 64, dtype=torch.bfloat16)
    far = torch.zeros(2**32 + 256, dtype=torch.bfloat16, device="cuda").as_strided((2, 2, 64), (2**31, 2**30, 1))
    far.copy_(x)
    out = torch.zeros(2**32 + 256, dtype=torch.bfloat16, device="cuda").as_strided((2, 2, 64), (2**31, 2**30, 1))
    for over in ("token", "sequence"):
        ref = dc.dynconv_groupnorm_fwd(x, 2, over=over)
        assert torch.equal(dc.dynconv_groupnorm_fwd(far, 2, over=over, out=out), ref)
        assert torch.equal(dc.dynconv_groupnorm_bwd(far, 2, x, over=over)[0], dc.dynconv_groupnorm_bwd(x, 2, x, over=over)[0])


def test_empty():
    x, w = torch.zeros(0, 5, 64, device="cuda"), torch.ones(64, device="cuda")
    for over in ("token", "sequence"):
        for t in (x, x.reshape(5, 0, 64)):
            y, stats = dc.dynconv_groupnorm_fwd(t, 4, w, w, over=over, want_stats=True)
            assert y.shape == t.shape
            if stats is not None:
                assert stats.shape == (t.shape[0], 4, 2) and not stats.any()
            dx, dw, db, _ = dc.dynconv_groupnorm_bwd(t, 4, t, w, w, over=over)
            assert dx.shape == t.shape and float(dw.abs().max()) == 0.0 == float(db.abs().max())


def test_gradients_are_differences():
    """Central differences of the kernels' own forward in float32. Allowed: what the oracle's difference of
    the same step is off from its gradient, and the forward's error bound over the step."""
    for over in ("token", "sequence"):
        x, gate, dy = rand(120, 2, 6, 24), rand(121, 2, 6, 24), rand(122, 2, 6, 24)
        w, bias = 1 + rand(123, 24, scale=0.1), rand(124, 24)
        t = {"x": x, "weight": w, "bias": bias, "gate": gate}
        t64 = {n: to64(v) for n, v in t.items()}
        kw = dict(activation="silu", over=over)
        got = dict(zip(("x", "weight", "bias", "gate"), dc.dynconv_groupnorm_bwd(x, 3, dy, w, bias, gate, **kw)))
        exact = dict(zip(("x", "weight", "bias", "gate"), groupnorm_bwd(t64["x"], 3, to64(dy), t64["weight"], t64["bias"], t64["gate"], **kw)))
        h = 2.0**-5
        noise = 1.5 * (np.abs(to64(dy)) * (bounds(t64["x"], 3, to64(dy), t64["weight"], t64["bias"], t64["gate"], **kw)[0]
                                           + U * np.abs(groupnorm_fwd(t64["x"], 3, t64["weight"], t64["bias"], t64["gate"], **kw)))).sum() / h

        def loss():
            return float((dc.dynconv_groupnorm_fwd(t["x"], 3, t["weight"], t["bias"], t["gate"], **kw).double() * dy.double()).sum())

        def loss64():
            return float((groupnorm_fwd(t64["x"], 3, t64["weight"], t64["bias"], t64["gate"], **kw) * to64(dy)).sum())

        def difference(v, at, value):
            keep = float(v[at])
            v[at] = np.float32(keep + h).item()
            up, hi = value(), float(v[at])
            v[at] = np.float32(keep - h).item()
            down, lo = value(), float(v[at])
            v[at] = keep
            return (up - down) / (hi - lo)

        for name, at in (("x", (0, 2, 5)), ("x", (1, 5, 23)), ("weight", (9,)), ("bias", (0,)), ("gate", (1, 0, 12))):
            off = abs(difference(t64[name], at, loss64) - exact[name][at])
            assert abs(difference(t[name], at, loss) - float(got[name][at])) <= 1.01 * off + noise, (over, name, at)


def test_same_bits_every_time_captured_and_on_other_streams():
    x, gate, dy = (rand(130 + i, 2, 900, 256, dtype=torch.bfloat16) for i in range(3))
    w = rand(133, 256, dtype=torch.bfloat16)
    lengths = torch.tensor([900, 411], dtype=torch.int32, device="cuda")

    def work():
        out = []
        for kw in (dict(over="token"), dict(over="sequence", lengths=lengths)):
            y, stats = dc.dynconv_groupnorm_fwd(x, 8, w, w, gate, "silu", want_stats=True, **kw)
            out += [y, *dc.dynconv_groupnorm_bwd(x, 8, dy, w, w, gate, "silu", stats=stats, **kw)]
            out += list(dc.dynconv_groupnorm_bwd(dc.dynconv_pack8(x), 8, dy, w, w, gate, "silu", **kw))
        return out

    first = work()
    assert all(torch.equal(a, b) for a, b in zip(first, work()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(4):
        x.copy_(rand(140 + i, 2, 900, 256))
        lengths.copy_(torch.tensor([900 - 100 * i, 411 + 7 * i]))
        eager = work()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        other = work()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, eager))


def test_refusals():
    x, w = rand(150, 2, 4, 64), rand(151, 64)
    with pytest.raises(DynconvError, match="INVALID_ARG"):
        dc.dynconv_groupnorm_fwd(x, 4, w, out=x)
    with pytest.raises(DynconvError, match="INVALID_ARG"):
        dc.dynconv_groupnorm_fwd(x, 4, w, eps=-1.0)
    with pytest.raises(DynconvError, match="UNSUPPORTED"):
        dc.dynconv_groupnorm_fwd(rand(152, 2, 64, 4).transpose(1, 2), 4)
    with pytest.raises(RuntimeError):
        dc.dynconv_groupnorm_fwd(x, 4, w.cpu())
    for bad in (dict(groups=5), dict(groups=0), dict(groups=4, over="batch"), dict(groups=4, activation="relu"),
                dict(groups=4, lengths=torch.ones(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            dc.dynconv_groupnorm_fwd(x, **bad)


def test_more_groups_than_one_dimension_of_a_launch():
    """2^26 (sequence, group) pairs: the waves that finish their statistics are more than 2^32 threads."""
    B, groups = 2**20 + 3, 64
    x = torch.ones(B, 1, 2 * groups, dtype=torch.bfloat16, device="cuda")
    x[..., 1::2] = 3.0
    x[-5:] = rand(160, 5, 1, 2 * groups, dtype=torch.bfloat16)
    y = dc.dynconv_groupnorm_fwd(x, groups, over="sequence")
    ref = groupnorm_fwd(to64(x[-8:]), groups, over="sequence")
    near("last rows", y[-8:], ref, bounds(to64(x[-8:]), groups, np.zeros((8, 1, 2 * groups)), over="sequence")[0])
    assert bool((y[:-5, :, 0::2] == y[0, 0, 0]).all()) and bool((y[:-5, :, 1::2] == y[0, 0, 1]).all())
