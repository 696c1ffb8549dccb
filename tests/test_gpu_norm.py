"""GPU parity of the RMS norm with weight, SiLU gate and scaled residual against the float64
oracle, through the C ABI.

Tolerances: a 16-bit result is rounded once (rtol 2^-8 bf16, 2^-11 float16); float32 arithmetic
in front of it is good to a few 2^-24 of the value and, in the backward's difference of two
terms, of the largest value (parity.assert_close's atol). dweight sums rows in float32: at most
rows / 1024 + 16 roundings of a running sum per partial, the partials in float64: 1e-5.
"""
import numpy as np
import pytest
import torch

from dynamic_short_convolution_amd import DynconvError, dynconv_norm_bwd, dynconv_norm_fwd
from oracle import norm_bwd, norm_fwd
from tests.parity import assert_close, to64

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    yield
    torch.cuda.synchronize()


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    return (torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)) * scale).to(dtype).cuda()


def check(shape, dtype, gated, at, weighted=True, alpha=0.37, eps=1e-5, dh=True):
    td = TD[dtype]
    x, dy = rand(1, *shape, dtype=td), rand(2, *shape, dtype=td)
    w = (1 + rand(3, shape[-1], scale=0.1)).to(td) if weighted else None
    z = rand(4, *shape, dtype=td) if gated else None
    r = rand(5, *shape, dtype=td, scale=3.0) if at else None
    gh = rand(6, *shape, dtype=td) if at == "before" and dh else None
    opt = lambda t: None if t is None else to64(t)  # noqa: E731
    kw = dict(gate=z, residual=r, residual_scale=alpha, eps=eps)
    out = dynconv_norm_fwd(x, w, residual_at=at or "before", **kw)
    xin = to64(x)
    if at == "before":
        y, h = out
        # the stream's sum in float32 arithmetic, then the storage type: the same bits as torch's
        assert torch.equal(h, (r.float() + alpha * x.float()).to(td))
        xin = to64(h)
    else:
        y, h = out, x
    ref = norm_fwd(xin, opt(w), opt(z), eps)
    up = np.float32(alpha).astype(np.float64)
    assert_close("y", y, to64(r) + up * ref if at == "after" else ref, td)
    dx, dres, dw, dz = dynconv_norm_bwd(h, w, dy, gate=z, dh=gh, residual_scale=alpha, residual_at=at, eps=eps)
    rx, rw, rz = norm_bwd(xin, opt(w), opt(z), to64(dy) * (up if at == "after" else 1.0), eps)
    if at == "before":
        rx = rx + (to64(gh) if gh is not None else 0.0)
        assert_close("dresidual", dres, rx, td)
        rx = up * rx
    else:
        assert dres is None
    assert_close("dx", dx, rx, td)
    assert (dw is None) == (w is None) and (dz is None) == (z is None)
    if w is not None:
        assert dw.dtype == torch.float32
        assert_close("dweight", dw, rw, torch.float32, rtol=1e-5, atol=1e-5)
    if z is not None:
        assert_close("dgate", dz, rz, td)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gated,at", [(False, None), (True, None), (False, "before"), (True, "before"), (False, "after"),
                                      (True, "after")])
@pytest.mark.parametrize("shape", [(300, 128), (37, 1), (5, 2, 64), (70, 100), (33, 515), (9, 2, 3, 256), (20, 2048), (7, 1537),
                                   (3, 8192), (2, 9000), (3, 20001), (40, 4096)], ids=str)
def test_against_oracle(shape, gated, at, dtype):
    check(shape, dtype, gated, at)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_without_weight_or_dh(dtype):
    check((50, 96), dtype, True, None, weighted=False)
    check((50, 96), dtype, False, "before", weighted=False, dh=False)
    check((2, 9000), dtype, True, "before", weighted=False, dh=False)


@pytest.mark.parametrize("rows", [1, 2, 17, 5000, 40000])
def test_weight_gradient_over_many_rows(rows):
    check((rows, 64), "bf16", True, None)
    check((max(1, rows // 8), 2048), "bf16", False, "before")


def test_empty():
    x = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    assert dynconv_norm_fwd(x, w).shape == (0, 64)
    dx, _, dw, _ = dynconv_norm_bwd(x, w, x)
    assert dx.shape == (0, 64) and float(dw.abs().max()) == 0.0
    assert dynconv_norm_fwd(torch.zeros(5, 0, device="cuda")).shape == (5, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_zero_and_large_rows(dtype):
    td = TD[dtype]
    x = torch.zeros(4, 128, dtype=td, device="cuda")
    x[1], x[2], x[3, 5] = 1e15, 1e-15, 3.0
    y = dynconv_norm_fwd(x, eps=1e-6)
    assert bool(torch.isfinite(y).all()) and float(y[0].abs().max()) == 0.0
    assert_close("y", y, norm_fwd(to64(x), None, None, 1e-6), td)
    x[0, 3] = float("nan")
    y2 = dynconv_norm_fwd(x, eps=1e-6)
    assert bool(y2[0].isnan().all()) and torch.equal(y2[1:], y[1:])


def test_large_gates():
    """SiLU of large arguments: 0 and z, no overflow."""
    x, z = rand(7, 4, 64), torch.tensor([-1e4, -100.0, 100.0, 1e4], device="cuda")[:, None].expand(4, 64)
    with pytest.raises(DynconvError, match="UNSUPPORTED"):  # one value for a whole row: not adjacent channels
        dynconv_norm_fwd(x, gate=z)
    z = z.contiguous()
    y = dynconv_norm_fwd(x, gate=z)
    assert_close("y", y[2:], norm_fwd(to64(x), None, to64(z))[2:], torch.float32)
    assert float(y[:2].abs().max()) < 1e-30
    dz = dynconv_norm_bwd(x, None, x, gate=z)[3]
    assert bool(torch.isfinite(dz).all())


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 63), ("f32", 64), ("f16", 200)])
def test_strided_views_inside_guard_bands(dtype, D):
    td = TD[dtype]
    shape = (3, 5, 4, D)

    def inside(t, off):
        big = torch.full((t.shape[2] + 1, t.shape[0] + 1, t.shape[1] + 2, D + 16 + off), float("nan"), dtype=td, device="cuda")
        v = big[:-1, 1:, 1:-1, off:off + D].permute(1, 2, 0, 3)
        v.copy_(t)
        return big, v

    x, z, r, dy, dh = (rand(10 + i, *shape, dtype=td) for i in range(5))
    w = rand(20, D, dtype=td)
    ref = dynconv_norm_fwd(x, w, gate=z, residual=r, residual_scale=0.5)
    for off in (0, 1):
        views = [inside(t, off)[1] for t in (x, z, r, dy, dh)]
        bo, o = inside(torch.zeros_like(x), off)
        bh, h = inside(torch.zeros_like(x), off)
        dynconv_norm_fwd(views[0], w, gate=views[1], residual=views[2], residual_scale=0.5, out=o, out_h=h)
        assert torch.equal(h, ref[1]) and int(torch.isfinite(bo).sum()) == x.numel() == int(torch.isfinite(bh).sum())
        assert_close("y", o, to64(ref[0]), td)
        a = dynconv_norm_bwd(h, w, views[3], gate=views[1], dh=views[4], residual_scale=0.5, residual_at="before")
        b = dynconv_norm_bwd(ref[1], w, dy, gate=z, dh=dh, residual_scale=0.5, residual_at="before")
        for name, s, t in zip(("dx", "dres", "dw", "dz"), a, b):
            assert_close(name, s, to64(t), t.dtype, rtol=1e-5 if name == "dw" else None, atol=1e-5 if name == "dw" else None)


def test_offsets_past_32_bits():
    x = rand(30, 2, 64, dtype=torch.bfloat16)
    far = torch.zeros(2**31 + 64, dtype=torch.bfloat16, device="cuda").as_strided((2, 64), (2**31, 1))
    far.copy_(x)
    assert torch.equal(dynconv_norm_fwd(far), dynconv_norm_fwd(x))
    out = torch.zeros(2**31 + 64, dtype=torch.bfloat16, device="cuda").as_strided((2, 64), (2**31, 1))
    assert torch.equal(dynconv_norm_fwd(x, out=out), dynconv_norm_fwd(x))


def test_more_rows_than_one_dimension_of_a_launch():
    """2^23 workgroups of 16 rows are one dimension's; the rows behind them are the second's."""
    n = 2**27 + 37
    x = torch.full((n, 1), 2.0, dtype=torch.bfloat16, device="cuda")
    x[-37:, 0] = torch.arange(1, 38, device="cuda").to(torch.bfloat16)
    y = dynconv_norm_fwd(x, eps=1.0)
    part = x[-64:].double()
    ref = part / (part * part + 1.0).sqrt()
    assert bool(((y[-64:].double() - ref).abs() <= 2.0**-8 * ref).all())
    assert bool((y[:-37] == y[0]).all())


def test_captured_replayed_and_on_other_streams():
    x, z, w = rand(40, 3000, 128, dtype=torch.bfloat16), rand(41, 3000, 128, dtype=torch.bfloat16), rand(42, 128, dtype=torch.bfloat16)

    def work():
        y = dynconv_norm_fwd(x, w, gate=z)
        dx, _, dw, dz = dynconv_norm_bwd(x, w, y, gate=z)
        return [y, dx, dw, dz]

    work()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = work()
    for i in range(4):
        x.copy_(rand(50 + i, 3000, 128))
        eager = work()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = work()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, eager))


def test_refusals():
    x, w = rand(60, 4, 64), rand(61, 64)
    with pytest.raises(DynconvError, match="INVALID_ARG"):
        dynconv_norm_fwd(x, w, out=x)
    with pytest.raises(DynconvError, match="INVALID_ARG"):
        dynconv_norm_fwd(x, w, eps=-1.0)
    with pytest.raises(DynconvError, match="UNSUPPORTED"):
        dynconv_norm_fwd(rand(62, 64, 4).t(), None)
    with pytest.raises(RuntimeError):
        dynconv_norm_fwd(x, w.cpu())
    buf = torch.zeros(64, device="cuda")
    with pytest.raises(DynconvError, match="INVALID_ARG"):
        dynconv_norm_fwd(x, w, out=buf.expand(4, 64))
