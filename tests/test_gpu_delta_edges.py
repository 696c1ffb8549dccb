"""Edges of the gated delta rule on the GPU: the split of operands into terms, vectors without an
epsilon, a single token with strides that mean nothing."""
import numpy as np
import pytest
import torch

from dynamic_short_convolution_amd import _lib, dynconv_delta_bwd, dynconv_delta_fwd, dynconv_delta_step
from oracle import delta_bwd, delta_fwd
from tests.parity import to64
from tests.test_gpu_delta import EPS, TD, check, close, documents, make, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    yield
    torch.cuda.synchronize()


def shrink(got, ref):
    """What share of the results is missing, on average: -<got - ref, ref> / <ref, ref>."""
    return -float(np.sum((to64(got) - ref) * ref) / np.sum(ref * ref))


def test_sixteen_bit_results_are_not_shrunk():
    """Operands that only reach float16 results are held in two terms of 8 bits. Rounded to nearest,
    what they leave out has either sign, as has the rounding of the results, which is the larger
    (at most 2^-11 of a value, 2^-12 in the root mean square): over N results its part along them
    is about 2^-12 / sqrt(N), with N > 2^18 2^-21, and ten of these are under 2^-17.5. Terms cut
    off instead leave out 2^-17 of a factor on average, all of one sign, and the product of the two
    second terms is 2^-17 on average: a product P U then lacks 3 * 2^-17, 2^-15.4."""
    B, T, Hk, Hv, dk, dv = 2, 300, 4, 4, 128, 128
    args = make(101, B, T, Hk, Hv, dk, dv, "f16")
    do = rand(102, B, T, Hv, dv, dtype=torch.float16)
    a64 = [to64(a) for a in args]
    got = [dynconv_delta_fwd(*args, scale=0.3, qk_norm_eps=EPS), *dynconv_delta_bwd(*args, do, scale=0.3, qk_norm_eps=EPS)[:2]]
    ref = [delta_fwd(*a64, 0.3, EPS)[0], *delta_bwd(*a64, to64(do), 0.3, EPS)[:2]]
    lost = {n: shrink(g, r) for n, g, r in zip(("o", "dq", "dk"), got, ref)}
    assert all(abs(x) < 2.0**-17.5 for x in lost.values()), lost


# ---------------------------------------------------------------------------------
# Unit vectors without an epsilon
# ---------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(2, 1, 1, 2, 64, 48), (1, 63, 2, 2, 128, 32), (1, 65, 1, 2, 64, 64), (2, 130, 1, 1, 37, 51),
                                   (1, 577, 1, 2, 40, 24)], ids=lambda s: "x".join(map(str, s)))
def test_unit_vectors_without_epsilon(shape, dtype):
    """qk_norm_eps = 0 with rows that are not zero: what the tokens behind the last one in its chunk
    of 64 read as (zeros) must not be divided by their length. 577 tokens: several segments."""
    B, T, Hk, Hv, dk, dv = shape
    args = make(111, *shape, dtype)
    check(args, eps=0.0, state=rand(112, B, Hv, dk, dv), dstate_out=rand(113, B, Hv, dk, dv))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_one_token_without_epsilon_is_a_step(dtype):
    args = make(114, 2, 1, 1, 2, 64, 80, dtype)
    S = rand(115, 2, 2, 64, 80)
    o, last = dynconv_delta_fwd(*args, qk_norm_eps=0.0, state=S, want_state=True)
    out = dynconv_delta_step(*[a[:, 0] for a in args], S, qk_norm_eps=0.0)
    ro, rl = delta_fwd(*[to64(a) for a in args], 0.125, 0.0, None, to64(rand(115, 2, 2, 64, 80)))
    for name, got, ref in (("o", o, ro), ("one step's o", out, ro[:, 0]), ("state", last, rl), ("one step's state", S, rl)):
        close(name, got, ref, TD[dtype])


# ---------------------------------------------------------------------------------
# One token: its stride has no meaning
# ---------------------------------------------------------------------------------


def one_token_strides(kind, H, d):
    """Strides of a [B, 1, H, d] tensor: channels first, an expanded row, far apart tokens."""
    return {"channels_first": (H * d, 1, d, 1), "expanded": (H * d, 0, d, 1), "short": (H * d, 8, d, 1),
            "far": (H * d, 2**26, d, 1), "farther": (H * d, 2**31, d, 1)}[kind]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["channels_first", "expanded", "short", "far", "farther"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (37, 51)])
def test_one_token_of_any_stride(kind, dk, dv, dtype):
    """Inputs, outputs and gradients of one token, bit for bit those of contiguous ones, inside guard
    bands."""
    B, H = 2, 2
    args = make(121, B, 1, H, H, dk, dv, dtype)
    do, state, ds = rand(122, B, 1, H, dv, dtype=TD[dtype]), rand(123, B, H, dk, dv), rand(124, B, H, dk, dv)

    def view(t):
        """A copy of t [B, 1, H, d] with such strides, between NaN."""
        d = t.shape[-1]
        big = torch.full((8 + B * H * d + 8,), float("nan"), dtype=t.dtype, device="cuda")
        v = big.as_strided((B, 1, H, d), one_token_strides(kind, H, d), 8)
        v.copy_(t)
        return big, v

    views = [view(a)[1] for a in args[:3]] + args[3:]
    kw = dict(qk_norm_eps=EPS, state=state)
    ref, last = dynconv_delta_fwd(*args, want_state=True, **kw)
    big, out = view(torch.zeros_like(ref))
    assert out.stride()[1] == one_token_strides(kind, H, dv)[1]
    got = dynconv_delta_fwd(*views, out=out, want_state=True, **kw)
    assert torch.equal(out, ref) and torch.equal(got[1], last) and int(torch.isfinite(big).sum()) == out.numel()
    assert torch.equal(dynconv_delta_step(*[a[:, 0] for a in views], state.clone(), qk_norm_eps=EPS),
                       dynconv_delta_step(*[a[:, 0] for a in args], state.clone(), qk_norm_eps=EPS))

    grads = dynconv_delta_bwd(*args, do, dstate_out=ds, need_dstate=True, **kw)
    vdo = view(do)[1]
    same = dynconv_delta_bwd(*views, vdo, dstate_out=ds, need_dstate=True, **kw)
    assert all(torch.equal(a, b) for a, b in zip(grads, same))
    # the gradients written with such strides, through the C entry point
    sp = lambda t: (t.data_ptr(), _lib.strides(t.stride()))  # noqa: E731
    outs = [view(torch.zeros_like(t)) for t in grads[:3]]
    dg, db, dst = (torch.zeros_like(t) for t in grads[3:])
    size = _lib.load().dynconv_delta_bwd_workspace_size(B, 1, H, H, dk, dv, {"f32": 0, "bf16": 1, "f16": 2}[dtype])
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    _lib.check("dynconv_delta_bwd", _lib.load().dynconv_delta_bwd(
        *(x for t in views for x in sp(t)), None, None, *sp(state), *sp(vdo), *sp(ds), *(x for _, t in outs for x in sp(t)),
        *sp(dg), *sp(db), *sp(dst), B, 1, H, H, dk, dv, dk**-0.5, EPS, {"f32": 0, "bf16": 1, "f16": 2}[dtype], work.data_ptr(), size,
        torch.cuda.current_stream().cuda_stream))
    assert all(torch.equal(a, b) for a, b in zip([t for _, t in outs] + [dg, db, dst], grads))
    assert all(int(torch.isfinite(b).sum()) == t.numel() for b, t in outs)


# ---------------------------------------------------------------------------------
# Broadcast inputs
# ---------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (37, 51), (128, 40)])
@pytest.mark.parametrize("shared", ["q", "k", "v", "g", "beta", "do", "state", "all"])
def test_broadcast_inputs_are_their_copies(shared, dk, dv, dtype):
    """Inputs with strides of 0, over sequences, tokens or heads, against contiguous copies: the same
    values through the same kernels, so the same bits. One row of k for all tokens takes the kernels
    for overlapping rows, whose float32 sums of the same terms may be contracted differently: each side's
    are within 4e-6 of the largest of the exact ones (dg 1e-5), and rounding puts each off by at
    most half a step."""
    B, T, H = 2, 80, 2
    args = make(131, B, T, H, H, dk, dv, dtype) + [rand(132, B, T, H, dv, dtype=TD[dtype]), rand(133, B, H, dk, dv)]
    names = ["q", "k", "v", "g", "beta", "do", "state"]
    over = [0, 1, 2, 2, 1, 0, 0]  # the dimension that is broadcast
    sizes = [a.shape for a in args]
    ex = [a.narrow(d, 0, 1).expand(s) if shared in (n, "all") else a for n, a, d, s in zip(names, args, over, sizes)]
    full = [a.contiguous() for a in ex]
    assert any(0 in a.stride() for a in ex)

    def run(q, k, v, g, beta, do, state):
        o, last = dynconv_delta_fwd(q, k, v, g, beta, qk_norm_eps=EPS, state=state, want_state=True)
        return [o, last, *dynconv_delta_bwd(q, k, v, g, beta, do, qk_norm_eps=EPS, state=state, need_dstate=True)]

    for name, a, b in zip(("o", "state", "dq", "dk", "dv", "dg", "dbeta", "dstate"), run(*ex), run(*full)):
        if dk % 8 or shared not in ("k", "all"):
            assert torch.equal(a, b), name
            continue
        step = 0.0 if a.dtype == torch.float32 else torch.finfo(a.dtype).eps
        a, b = a.double(), b.double()
        off = (a - b).abs() - step * torch.maximum(a.abs(), b.abs())
        assert float(off.max()) <= 2 * (1e-5 if name == "dg" else 4e-6) * float(b.abs().max()), name


# ---------------------------------------------------------------------------------
# The decay's gradient stays in its document
# ---------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("decay", [None, -float("inf"), -200.0, -104.0])
def test_decay_gradient_stays_in_its_document(decay, dtype):
    """Two documents in one row (or a token whose decay is 0 in float32 in the start's place), the second
    without a gradient of its own: every gradient of it is 0, not what is left of the first one's
    sums when they are taken off again."""
    B, T, H, dk, dv, start = 1, 100, 2, 64, 64, 41
    args = make(141, B, T, H, H, dk, dv, dtype)
    args[3][:, 5, 0] = -104.5
    seq = None
    if decay is None:
        seq = (torch.arange(T, device="cuda", dtype=torch.int32) >= start).to(torch.int32).expand(B, T).contiguous()
    else:
        args[3][:, start] = decay
    do = rand(142, B, T, H, dv, dtype=TD[dtype])
    do[:, start:] = 0.0
    check(args, seq=seq, do=do)
    grads = dynconv_delta_bwd(*args, do, qk_norm_eps=EPS, seq_idx=seq)
    for name, t in zip(("dq", "dk", "dv", "dg", "dbeta"), grads):
        assert float(t[:, :start].abs().max()) > 0.0 and float(t[:, start:].abs().max()) == 0.0, name
    assert float(grads[3][:, 5, 0].abs().max()) == 0.0  # exp(-104.5) is 0


# ---------------------------------------------------------------------------------
# Every instantiation of the kernels
# ---------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3])
@pytest.mark.parametrize("wide", [True, False], ids=["rows16", "elements"])
@pytest.mark.parametrize("T", [100, 580], ids=["whole", "segments"])
def test_every_instantiation(T, wide, group, dk, dtype):
    """Each storage type, padded key width, way of loading rows, and head grouping, over one scan and
    over segments, forwards and backwards, against the oracle."""
    B, Hk, dv = 1, 1, 40
    args = make(151, B, T, Hk, Hk * group, dk, dv, dtype, decay=0.3)
    if not wide:  # one element off a 16-byte boundary
        for i in range(3):
            off = torch.zeros(args[i].numel() + 1, dtype=args[i].dtype, device="cuda")[1:].view(args[i].shape)
            args[i] = off.copy_(args[i])
    H = Hk * group
    check(args, seq=documents(152, B, T, 70), state=rand(153, B, H, dk, dv), dstate_out=rand(154, B, H, dk, dv))
