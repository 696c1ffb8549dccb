"""GPU parity of the gated delta rule against the float64 oracle, through the C ABI.

Tolerances. A 16-bit result is rounded once (half a step: 2^-8 bf16, 2^-11 float16 relative to
the value, the rtol below) and its products keep two 8-bit terms per operand (2^-16 of each
factor, truncated): 2^-15 of the sum of |terms|, taken as at most twice the largest result:
atol = 2^-14 of max|ref|. Float32 results (states, dg, float32 storage) are sums of products
held to 2^-23 each, over 64 tokens, up to 128 channels and a chain of chunks that forgets:
atol = 64 * 2^-24 = 4e-6 of max|ref|; dg adds the cumulative sum over a chunk of 64 such terms:
sqrt(64) more in the worst direction taken as 2.5 times: 1e-5.
"""
import numpy as np
import pytest
import torch

from dynamic_short_convolution_amd import (DynconvError, dynconv_cache_fill, dynconv_decode_step, dynconv_delta_bwd,
                                           dynconv_delta_fwd, dynconv_delta_step, dynconv_fwd, dynconv_bwd,
                                           dynconv_norm_bwd, dynconv_norm_fwd, new_delta_state)
from oracle import conv_bwd, conv_fwd, delta_bwd, delta_fwd, norm_bwd, norm_fwd
from tests.parity import assert_close, rel_max_err, to64

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dstate")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    yield
    torch.cuda.synchronize()


def close(name, got, ref, dtype, scale=1.0, extra=None):
    f32 = got.dtype == torch.float32
    atol = (1e-5 if name == "dg" else 4e-6) if f32 else 2.0**-14
    if float(np.max(np.abs(ref), initial=0.0)) == 0.0:
        assert float(got.abs().max()) <= 1e-6 * scale, name
        return
    assert_close(name, got, ref, got.dtype, atol=atol * scale, extra=extra)


def make(seed, B, T, Hk, Hv, dk, dv, dtype, norm=True, decay=1.0):
    rng = np.random.default_rng([seed, B, T, dk, dv])
    td = TD[dtype]

    def n(*shape):
        return rng.standard_normal(shape)

    q, k = n(B, T, Hk, dk), n(B, T, Hk, dk) + 0.5
    if not norm:
        q, k = (a / np.sqrt(np.sum(a * a, -1, keepdims=True)) for a in (q, k))
    t = lambda a, d=td: torch.from_numpy(a).to(d).cuda()  # noqa: E731
    return [t(q), t(k), t(n(B, T, Hv, dv)), t(-decay * np.abs(n(B, T, Hv)) * 0.3, torch.float32),
            t(1 / (1 + np.exp(-n(B, T, Hv))))]


def documents(seed, B, T, mean):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(np.cumsum(rng.random((B, T)) < 1.0 / mean, axis=1).astype(np.int32)).cuda()


def rand(seed, *shape, dtype=torch.float32):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)).to(dtype).cuda()


def check(args, scale=0.3, eps=EPS, seq=None, state=None, dstate_out=None, do=None, backward=True):
    B, T, Hv, dv = args[2].shape
    dtype = args[0].dtype
    do = rand(999, B, T, Hv, dv, dtype=dtype) if do is None else do
    a64 = [to64(a) for a in args]
    s64 = None if seq is None else seq.cpu().numpy()
    st64 = None if state is None else to64(state)
    o, last = dynconv_delta_fwd(*args, scale=scale, qk_norm_eps=eps, seq_idx=seq, state=state, want_state=True)
    ro, rl = delta_fwd(*a64, scale, eps, s64, st64)
    close("o", o, ro, dtype)
    close("state", last, rl, torch.float32)
    if not backward:
        return
    got = dynconv_delta_bwd(*args, do, scale=scale, qk_norm_eps=eps, seq_idx=seq, state=state, dstate_out=dstate_out,
                            need_dstate=True)
    ref = delta_bwd(*a64, to64(do), scale, eps, s64, st64, None if dstate_out is None else to64(dstate_out))
    # The norm's gradient is (d - q^ (q^.d)) / |q|: what is left can be far smaller than d (with
    # one channel it is d eps / |q|^2), but its rounding errors are those of d / |q|, 4e-6 of it.
    extra = [None] * 6
    if eps is not None:
        unit, lens = zip(*((a / n, n) for a, n in ((a, np.sqrt(np.sum(a * a, -1, keepdims=True) + eps)) for a in a64[:2])))
        before = delta_bwd(*unit, *a64[2:], to64(do), scale, None, s64, st64, None if dstate_out is None else to64(dstate_out))
        extra[:2] = [4e-6 * np.sqrt(np.sum(d * d, -1, keepdims=True)) / n * np.ones_like(d) for d, n in zip(before[:2], lens)]
    for name, g, r, x in zip(GRADS, got, ref, extra):
        close(name, g, r, dtype, extra=x)


SHAPES = [  # B, T, Hk, Hv, dk, dv
    (1, 1, 1, 1, 8, 8), (2, 1, 2, 4, 128, 128), (1, 63, 1, 2, 64, 64), (2, 64, 1, 1, 128, 16), (1, 65, 2, 2, 128, 128),
    (1, 130, 1, 3, 32, 48), (2, 129, 2, 4, 96, 80), (1, 200, 1, 1, 120, 200), (1, 70, 3, 3, 37, 51), (3, 66, 1, 2, 1, 1),
    (1, 100, 1, 1, 65, 17), (1, 90, 2, 8, 64, 32),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_oracle(shape, dtype):
    B, T, Hk, Hv, dk, dv = shape
    args = make(1, *shape, dtype)
    check(args, seq=documents(5, B, T, 20), state=rand(2, B, Hv, dk, dv), dstate_out=rand(3, B, Hv, dk, dv))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("norm,state,docs", [(False, False, 0), (False, True, 30), (True, False, 0), (True, False, 3)])
def test_options(dtype, norm, state, docs):
    B, T, Hk, Hv, dk, dv = 2, 140, 1, 2, 64, 48
    args = make(11, B, T, Hk, Hv, dk, dv, dtype, norm)
    check(args, eps=EPS if norm else None, seq=documents(6, B, T, docs) if docs else None,
          state=rand(4, B, Hv, dk, dv) if state else None)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape,docs", [((1, 1600, 1, 1, 24, 16), 0), ((2, 1543, 1, 2, 16, 20), 300), ((1, 2100, 1, 1, 72, 16), 0)])
def test_long_sequences_in_segments(shape, docs, dtype):
    """Few heads, many chunks: the scans run over segments that are joined afterwards."""
    B, T, Hk, Hv, dk, dv = shape
    args = make(12, *shape, dtype, decay=0.05)  # slow decay: segments depend on one another
    check(args, seq=documents(8, B, T, docs) if docs else None, state=rand(5, B, Hv, dk, dv), dstate_out=rand(6, B, Hv, dk, dv))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [448, 449, 577])
def test_shortest_segments(T, dtype):
    """7 chunks (one segment), 8 (four of two) and 10 (four of two and the last of one)."""
    args = make(31, 1, T, 1, 2, 40, 24, dtype, decay=0.05)
    check(args, state=rand(32, 1, 2, 40, 24), dstate_out=rand(33, 1, 2, 40, 24))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_gates(dtype):
    """No write (beta 0), no decay, decays to zero (-inf, -1e30, below float32's exp), long sums
    of strong decays next to weak ones."""
    B, T, H, dk, dv = 1, 150, 2, 32, 32
    args = make(13, B, T, H, H, dk, dv, dtype)
    g, beta = args[3], args[4]
    beta[:, 10:20] = 0.0
    beta[:, 130:] = 1.0
    g[:, 30:60] = 0.0
    g[:, 70, 0], g[:, 71, 1], g[:, 90, 0], g[:, 64, 1] = -float("inf"), -1e30, -200.0, -127.0
    g[:, 100:125, 1] = -60.0
    g[:, 112, 1] = -1e-3
    check(args, state=rand(7, B, H, dk, dv), dstate_out=rand(8, B, H, dk, dv))


def test_all_writes_off_keeps_the_state():
    args = make(14, 2, 100, 1, 2, 64, 64, "bf16")
    args[3].zero_()
    args[4].zero_()
    S = rand(9, 2, 2, 64, 64)
    o, last = dynconv_delta_fwd(*args, qk_norm_eps=EPS, state=S, want_state=True)
    assert torch.equal(last, S)
    grads = dynconv_delta_bwd(*args, torch.randn_like(o), qk_norm_eps=EPS, state=S, need_dstate=True)
    assert float(grads[2].abs().max()) == 0.0  # dv = beta ...
    assert all(bool(torch.isfinite(t).all()) for t in grads)


def test_zero_rows_are_fine():
    """Zero q and k rows (a zero vector under the norm) give zeros, not NaN."""
    args = make(15, 1, 70, 1, 1, 32, 32, "bf16")
    args[0][:, 5:9] = 0.0
    args[1][:, 30:40] = 0.0
    check(args, eps=1e-3)
    o = dynconv_delta_fwd(*args, qk_norm_eps=1e-3)
    assert float(o[:, 5:9].abs().max()) == 0.0


def test_padding_behind_the_sequence():
    """Tokens with beta = 0 and g = 0 behind a sequence change nothing, bit for bit."""
    args = make(16, 2, 150, 1, 2, 128, 64, "bf16")
    o, last = dynconv_delta_fwd(*[a[:, :90] for a in args], qk_norm_eps=EPS, want_state=True)
    for a, val in ((args[3], 0.0), (args[4], 0.0)):
        a[:, 90:] = val
    o2, last2 = dynconv_delta_fwd(*args, qk_norm_eps=EPS, want_state=True)
    assert torch.equal(o2[:, :90], o) and torch.equal(last2, last)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_no_tokens(dtype):
    args = make(17, 2, 0, 1, 2, 16, 16, dtype)
    S = rand(10, 2, 2, 16, 16)
    o, last = dynconv_delta_fwd(*args, state=S, want_state=True)
    assert o.shape == (2, 0, 2, 16) and torch.equal(last, S)
    _, last = dynconv_delta_fwd(*args, want_state=True)
    assert float(last.abs().max()) == 0.0
    d = dynconv_delta_bwd(*args, o, state=S, dstate_out=2 * S, need_dstate=True)
    assert torch.equal(d[5], 2 * S) and d[0].shape == (2, 0, 1, 16)


@pytest.mark.parametrize("at", [3, 67])
def test_nan_stays_in_its_head(at):
    """A NaN reaches its head's chunk of 64 tokens and what follows, and nothing else."""
    args = make(18, 2, 130, 2, 2, 64, 64, "bf16")
    ref = dynconv_delta_fwd(*args, qk_norm_eps=EPS)
    args[2][1, at, 0, 5] = float("nan")
    o = dynconv_delta_fwd(*args, qk_norm_eps=EPS)
    assert torch.equal(o[0], ref[0]) and torch.equal(o[1, :, 1], ref[1, :, 1])
    assert bool(o[1, at:, 0, 5].isnan().all()) and torch.equal(o[1, :at // 64 * 64, 0], ref[1, :at // 64 * 64, 0])
    assert torch.equal(o[1, :, 0, :5], ref[1, :, 0, :5]) and torch.equal(o[1, :, 0, 6:], ref[1, :, 0, 6:])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (37, 51), (128, 40)])
def test_strided_views_inside_guard_bands(dtype, dk, dv):
    """Every tensor a view into a larger buffer of NaN: head-first inputs, padded rows, one
    element off a 16-byte boundary; outputs written nowhere else."""
    B, T, Hk, Hv = 2, 90, 2, 4
    args = make(19, B, T, Hk, Hv, dk, dv, dtype)

    def inside(t, order, off):
        """A copy of t whose memory order of dimensions is `order`, in a NaN buffer."""
        shape = [t.shape[i] for i in order]
        big = torch.full([n + 2 for n in shape[:-1]] + [shape[-1] + 8 + off], float("nan"), dtype=t.dtype, device="cuda")
        v = big[tuple(slice(1, 1 + n) for n in shape[:-1]) + (slice(off, off + shape[-1]),)]
        v = v.permute(*[order.index(i) for i in range(t.dim())])
        v.copy_(t)
        return big, v

    views = [inside(args[0], (0, 2, 1, 3), 1), inside(args[1], (0, 1, 2, 3), 0), inside(args[2], (2, 0, 1, 3), 3),
             inside(args[3], (2, 0, 1), 1), inside(args[4], (0, 2, 1), 1)]
    vargs = [v for _, v in views]
    seq = documents(21, B, T, 25)
    state = rand(20, B, Hv, dk, dv)
    ref = dynconv_delta_fwd(*args, qk_norm_eps=EPS, seq_idx=seq, state=state, want_state=True)
    big, out = inside(torch.zeros_like(ref[0]), (0, 2, 1, 3), 1)
    sbig, sout = inside(torch.zeros_like(state), (1, 0, 2, 3), 1)
    got = dynconv_delta_fwd(*vargs, qk_norm_eps=EPS, seq_idx=seq.t().contiguous().t(), state=inside(state, (1, 0, 2, 3), 3)[1],
                            out=out, state_out=sout)
    assert got[0] is out and got[1] is sout
    close("o", out, to64(ref[0]), TD[dtype])
    close("state", sout, to64(ref[1]), torch.float32)
    for buf, v in ((big, out), (sbig, sout)):
        assert int(torch.isfinite(buf).sum()) == v.numel()
    do = rand(22, B, T, Hv, dv, dtype=TD[dtype])
    ref = dynconv_delta_bwd(*args, do, qk_norm_eps=EPS, seq_idx=seq, state=state, need_dstate=True)
    got = dynconv_delta_bwd(*vargs, inside(do, (0, 2, 1, 3), 1)[1], qk_norm_eps=EPS, seq_idx=seq,
                            state=inside(state, (1, 0, 2, 3), 3)[1], need_dstate=True)
    for name, a, b in zip(GRADS, got, ref):
        close(name, a, to64(b), TD[dtype])


def test_broadcast_inputs():
    """Stride 0: gates shared by all heads, q and k shared by the batch, one row for all tokens."""
    B, T, H, dk, dv = 2, 80, 2, 64, 64
    q, k, v, g, b = make(23, B, T, H, H, dk, dv, "bf16")
    ex = [q[:1].expand(B, -1, -1, -1), k[:, :1].expand(-1, T, -1, -1), v[:, :, :1].expand(-1, -1, H, -1),
          g[..., :1].expand(-1, -1, H), b[:, :1].expand(-1, T, -1)]
    full = [t.contiguous() for t in ex]
    do = rand(24, B, T, H, dv, dtype=torch.bfloat16)
    for a, c in zip([dynconv_delta_fwd(*ex, qk_norm_eps=EPS), *dynconv_delta_bwd(*ex, do[:1].expand(B, -1, -1, -1), qk_norm_eps=EPS)[:5]],
                    [dynconv_delta_fwd(*full, qk_norm_eps=EPS), *dynconv_delta_bwd(*full, do[:1].repeat(B, 1, 1, 1), qk_norm_eps=EPS)[:5]]):
        assert rel_max_err(a, to64(c)) <= 2e-2


def test_offsets_past_32_bits():
    """Sequences 2^31 elements apart."""
    B, T, H, dk, dv = 2, 70, 1, 64, 64
    args = make(25, B, T, H, H, dk, dv, "bf16")
    ref = dynconv_delta_fwd(*args, qk_norm_eps=EPS)
    far = torch.zeros(2**31 + T * H * dk, dtype=torch.bfloat16, device="cuda")
    view = far.as_strided((B, T, H, dk), (2**31, H * dk, dk, 1))
    for i in range(3):
        moved = list(args)
        view.copy_(args[i])
        moved[i] = view
        assert torch.equal(dynconv_delta_fwd(*moved, qk_norm_eps=EPS), ref)
    out = dynconv_delta_fwd(*args, qk_norm_eps=EPS, out=view)
    assert torch.equal(out, ref)
    big = torch.zeros(2**31 + H * dk * dv, device="cuda")
    st = big.as_strided((B, H, dk, dv), (2**31, dk * dv, dv, 1))
    last = dynconv_delta_fwd(*args, qk_norm_eps=EPS, state_out=st)[1]
    assert torch.equal(last, dynconv_delta_fwd(*args, qk_norm_eps=EPS, want_state=True)[1])
    one = [a[:, 0] for a in args]
    c = st.clone()
    assert torch.equal(dynconv_delta_step(*one, st, qk_norm_eps=EPS), dynconv_delta_step(*one, c, qk_norm_eps=EPS))
    assert torch.equal(st, c)


def test_state_in_place():
    args = make(26, 2, 100, 1, 2, 64, 80, "bf16")
    S = rand(27, 2, 2, 64, 80)
    ref = dynconv_delta_fwd(*args, state=S, qk_norm_eps=EPS, want_state=True)
    o, last = dynconv_delta_fwd(*args, state=S, state_out=S, qk_norm_eps=EPS)
    assert last is S and torch.equal(o, ref[0]) and torch.equal(S, ref[1])


def test_state_in_place_over_segments():
    args = make(28, 1, 1700, 1, 1, 32, 16, "bf16", decay=0.05)
    S = rand(29, 1, 1, 32, 16)
    ref = dynconv_delta_fwd(*args, state=S, qk_norm_eps=EPS, want_state=True)
    o, _ = dynconv_delta_fwd(*args, state=S, state_out=S, qk_norm_eps=EPS)
    assert torch.equal(o, ref[0]) and torch.equal(S, ref[1])


def test_runs_are_identical():
    for shape in ((2, 300, 2, 4, 128, 128), (1, 1600, 1, 1, 64, 64)):
        args = make(30, *shape, "bf16")
        do = rand(31, shape[0], shape[1], shape[3], shape[5], dtype=torch.bfloat16)
        runs = [[dynconv_delta_fwd(*args, qk_norm_eps=EPS), *dynconv_delta_bwd(*args, do, qk_norm_eps=EPS, need_dstate=True)]
                for _ in range(3)]
        for r in runs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("Hk,Hv,dk,dv,norm", [(2, 2, 128, 128, True), (1, 3, 37, 51, True), (2, 4, 64, 40, False), (1, 1, 1, 1, True),
                                              (1, 2, 128, 200, True)])
def test_decoding_matches_the_whole_sequence(Hk, Hv, dk, dv, norm, dtype):
    """A prompt through the chunked form, then one token at a time."""
    B, T, T0 = 3, 80, 67
    args = make(33, B, T, Hk, Hv, dk, dv, dtype, norm)
    args[3][:, 70, 0] = -float("inf")
    eps = EPS if norm else None
    ro, rl = delta_fwd(*[to64(a) for a in args], 0.2, eps)
    o, state = dynconv_delta_fwd(*[a[:, :T0] for a in args], scale=0.2, qk_norm_eps=eps, want_state=True)
    close("prompt", o, ro[:, :T0], TD[dtype])
    pool = torch.full((B + 2, Hv + 1, dk, dv + 4), float("nan"), device="cuda")
    cache = pool[1:-1, :Hv, :, :dv]
    cache.copy_(state)
    for t in range(T0, T):
        out = dynconv_delta_step(*[a[:, t] for a in args], cache, scale=0.2, qk_norm_eps=eps)
        # one result's largest value can be far below its sequence's: bound by the sequence's
        assert rel_max_err(out, ro[:, t]) <= 2e-2 if dtype != "f32" else True
        assert np.max(np.abs(to64(out) - ro[:, t])) <= (2.0**-8 if dtype == "bf16" else 2.0**-11 if dtype == "f16" else 1e-5) * np.max(
            np.abs(ro))
    close("state", cache, rl, torch.float32)
    assert int(torch.isfinite(pool).sum()) == cache.numel()


def test_new_state_and_single_token():
    args = make(34, 2, 1, 1, 2, 64, 64, "f32")
    state = new_delta_state(2, 2, 64, 64, "cuda")
    o = dynconv_delta_step(*[a[:, 0] for a in args], state, qk_norm_eps=EPS)
    ref, last = dynconv_delta_fwd(*args, qk_norm_eps=EPS, want_state=True)
    close("o", o, to64(ref)[:, 0], torch.float32)
    close("state", state, to64(last), torch.float32)


def test_gradients_are_differences():
    """float32 kernel outputs, central differences along random directions: the loss is a sum of
    about 10^4 products held to 2^-22, a step of 2^-6 changes it by about 1, so the quotient is
    good to about 1e-3."""
    B, T, Hk, Hv, dk, dv = 1, 100, 1, 2, 16, 24
    args = make(35, B, T, Hk, Hv, dk, dv, "f32")
    state, do, ds = rand(36, B, Hv, dk, dv), rand(37, B, T, Hv, dv), rand(38, B, Hv, dk, dv)
    grads = dynconv_delta_bwd(*args, do, qk_norm_eps=1e-3, state=state, dstate_out=ds, need_dstate=True)

    def loss(a, s):
        o, last = dynconv_delta_fwd(*a, qk_norm_eps=1e-3, state=s, want_state=True)
        return float((o.double() * do.double()).sum() + (last.double() * ds.double()).sum())

    for i, grad in enumerate(grads):
        d = rand(40 + i, *grad.shape)
        d /= d.norm()
        h = 2.0**-6
        vals = []
        for sign in (1.0, -1.0):
            a, s = list(args), state
            if i < 5:
                a[i] = args[i] + sign * h * d
            else:
                s = state + sign * h * d
            vals.append(loss(a, s))
        num, ana = (vals[0] - vals[1]) / (2 * h), float((grad.double() * d.double()).sum())
        assert abs(num - ana) <= 2e-3 * max(1.0, abs(ana)), (GRADS[i], num, ana)


def test_other_stream():
    args = make(45, 2, 200, 1, 2, 64, 64, "bf16")
    do = rand(46, 2, 200, 2, 64, dtype=torch.bfloat16)
    ref = [dynconv_delta_fwd(*args, qk_norm_eps=EPS), *dynconv_delta_bwd(*args, do, qk_norm_eps=EPS)[:5]]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in side:  # two calls at once, each with its own workspace
        with torch.cuda.stream(s):
            got.append([dynconv_delta_fwd(*args, qk_norm_eps=EPS), *dynconv_delta_bwd(*args, do, qk_norm_eps=EPS)[:5]])
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, ref))


def test_captured_and_replayed():
    """Two graphs (training over segments, decoding) replayed in turn with eager work between:
    every replay equals the eager result on the inputs of the moment."""
    args = make(47, 1, 1600, 1, 1, 64, 64, "bf16", decay=0.05)
    do = rand(48, 1, 1600, 1, 64, dtype=torch.bfloat16)
    one = [a[:, 0].contiguous() for a in args]
    state = rand(49, 1, 1, 64, 64)

    def train():
        return [dynconv_delta_fwd(*args, qk_norm_eps=EPS), *dynconv_delta_bwd(*args, do, qk_norm_eps=EPS)[:5]]

    def decode():
        return [dynconv_delta_step(*one, state, qk_norm_eps=EPS)]

    train(), decode()
    torch.cuda.synchronize()
    graphs = []
    for fn in (train, decode):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = fn()
        graphs.append((g, out))
    for i in range(4):
        args[2].copy_(rand(50 + i, *args[2].shape))
        one[2].copy_(rand(60 + i, *one[2].shape))
        before = state.clone()
        eager = [t.clone() for t in train()]
        graphs[0][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], eager))
        graphs[1][0].replay()
        after = state.clone()
        state.copy_(before)
        o = decode()[0]
        torch.cuda.synchronize()
        assert torch.equal(graphs[1][1][0], o) and torch.equal(state, after)


def test_refusals():
    q, k, v, g, b = make(51, 1, 10, 1, 1, 16, 16, "bf16")
    with pytest.raises(RuntimeError):
        dynconv_delta_fwd(q, k.cpu(), v, g, b)
    with pytest.raises(DynconvError, match="INVALID_ARG"):
        dynconv_delta_fwd(q, k, v, g, b, out=v)
    wide = torch.zeros(1, 10, 1, 160, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(DynconvError, match="UNSUPPORTED"):
        dynconv_delta_fwd(wide, wide, v, g, b)
    with pytest.raises(DynconvError, match="UNSUPPORTED"):
        dynconv_delta_fwd(wide[..., ::10], k, v, g, b)  # channels not adjacent
    with pytest.raises(ValueError):
        dynconv_delta_fwd(q, k, v, g, b, seq_idx=torch.zeros(1, 9, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        dynconv_delta_fwd(q, k, v, g, b, seq_idx=torch.zeros(1, 10, dtype=torch.int64, device="cuda"))
    st = torch.zeros(1, 1, 16, 16, device="cuda")
    with pytest.raises(DynconvError, match="UNSUPPORTED"):
        dynconv_delta_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], b[:, 0], st.transpose(2, 3))
    one = [t[:, 0] for t in (q, k, v, g, b)]
    with pytest.raises(DynconvError, match="UNSUPPORTED"):
        dynconv_delta_step(*one, st[:, :, :, :1].expand(1, 1, 16, 16))
    with pytest.raises(DynconvError, match="INVALID_ARG"):
        dynconv_delta_step(*one, st[:, :, :1].expand(1, 1, 16, 16))  # every row in one place
    with pytest.raises(DynconvError, match="INVALID_ARG"):
        dynconv_delta_step(*one, st, out=v[:, 0])


# ---------------------------------------------------------------------------------
# A layer as it would be used: convolution, delta rule, gated norm
# ---------------------------------------------------------------------------------


def test_layer_forward_and_backward():
    """Short convolution on q, k, v, the gated delta rule, the gated norm, and all of it backwards,
    against the float64 oracles chained. float32 storage: each of the six calls is held to 1e-5
    of its largest value, so the chain to 6e-5."""
    B, T, H, d, W = 2, 150, 2, 32, 4
    D = H * d
    x = {n: rand(70 + i, B, T, D) for i, n in enumerate("qkv")}
    w = {n: rand(80 + i, B, T, D, W) * 0.3 for i, n in enumerate("qkv")}
    g, beta = -rand(90, B, T, H).abs() * 0.2, torch.sigmoid(rand(91, B, T, H))
    z, wn, dy = rand(92, B, T, H, d), 1 + 0.1 * rand(93, d), rand(94, B, T, H, d)
    seq = documents(95, B, T, 40)

    c = {n: dynconv_fwd(x[n], w[n], 1, seq_idx=seq).view(B, T, H, d) for n in "qkv"}
    o = dynconv_delta_fwd(c["q"], c["k"], c["v"], g, beta, qk_norm_eps=EPS, seq_idx=seq)
    y = dynconv_norm_fwd(o, wn, gate=z, eps=1e-5)
    do, _, dwn, dz = dynconv_norm_bwd(o, wn, dy, gate=z, eps=1e-5)
    dc = dynconv_delta_bwd(c["q"], c["k"], c["v"], g, beta, do, qk_norm_eps=EPS, seq_idx=seq)
    dx, dw = zip(*(dynconv_bwd(x[n], w[n], dc[i].view(B, T, D), 1, seq_idx=seq) for i, n in enumerate("qkv")))

    s = seq.cpu().numpy()
    c64 = {n: conv_fwd(to64(x[n]), to64(w[n]), 1, s).reshape(B, T, H, d) for n in "qkv"}
    scale = d**-0.5
    rest = (to64(g), to64(beta))
    o64 = delta_fwd(c64["q"], c64["k"], c64["v"], *rest, scale, EPS, s)[0]
    do64, dwn64, dz64 = norm_bwd(o64, to64(wn), to64(z), to64(dy), 1e-5)
    dc64 = delta_bwd(c64["q"], c64["k"], c64["v"], *rest, do64, scale, EPS, s)
    pairs = [("y", y, norm_fwd(o64, to64(wn), to64(z), 1e-5)), ("dweight", dwn, dwn64), ("dgate", dz, dz64), ("dg", dc[3], dc64[3]),
             ("dbeta", dc[4], dc64[4])]
    for i, n in enumerate("qkv"):
        rx, rw = conv_bwd(to64(x[n]), to64(w[n]), dc64[i].reshape(B, T, D), 1, s)
        pairs += [("dx " + n, dx[i], rx), ("dw " + n, dw[i], rw)]
    for name, got, ref in pairs:
        assert rel_max_err(got, ref) <= 6e-5, (name, rel_max_err(got, ref))


def test_layer_decoding():
    """Prompt, then tokens one at a time through the caches of the convolution and the delta rule:
    the same outputs as the whole sequence at once."""
    B, T, T0, H, d, W = 2, 30, 21, 2, 32, 4
    D = H * d
    x = {n: rand(100 + i, B, T, D) for i, n in enumerate("qkv")}
    w = {n: rand(110 + i, D, W) * 0.3 for i, n in enumerate("qkv")}
    g, beta = -rand(120, B, T, H).abs() * 0.2, torch.sigmoid(rand(121, B, T, H))
    z, wn = rand(122, B, T, H, d), 1 + 0.1 * rand(123, d)

    def conv(t0):
        return {n: dynconv_fwd(x[n][:, :t0].contiguous(), w[n]).view(B, t0, H, d) for n in "qkv"}

    c = conv(T)
    whole = dynconv_norm_fwd(dynconv_delta_fwd(c["q"], c["k"], c["v"], g, beta, qk_norm_eps=EPS), wn, gate=z)
    c = conv(T0)
    _, state = dynconv_delta_fwd(c["q"], c["k"], c["v"], g[:, :T0], beta[:, :T0], qk_norm_eps=EPS, want_state=True)
    caches = {n: dynconv_cache_fill(x[n][:, :T0], W) for n in "qkv"}
    for t in range(T0, T):
        c = {n: dynconv_decode_step(x[n][:, t], w[n], caches[n], t).view(B, H, d) for n in "qkv"}
        o = dynconv_delta_step(c["q"], c["k"], c["v"], g[:, t], beta[:, t], state, qk_norm_eps=EPS)
        y = dynconv_norm_fwd(o, wn, gate=z[:, t])
        assert rel_max_err(y, to64(whole[:, t])) <= 3e-5
