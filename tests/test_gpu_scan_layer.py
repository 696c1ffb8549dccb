"""The linear-recurrent layer as it is used: the short convolution, the gated linear scan behind it and the group norm
over its heads, trained (with the scan's and the norm's inputs kept whole, or in 8 bits), and decoded token by token
from the states that a prompt leaves.

Each operator is held to the float64 oracle of its own inputs in its own tests; here the chain is, stage by stage: every
stage's result against the oracle applied to what the stage before it gave, with the tolerances of tests/parity.py.
"""
import numpy as np
import pytest
import torch

import dynamic_short_convolution_amd as dc
import synth
from oracle import conv_bwd, groupnorm_bwd, groupnorm_fwd, held8, scan_bwd, scan_fwd
from tests.parity import assert_close, to64

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
W, HEADS = 4, 4


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    yield
    torch.cuda.synchronize()


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    return (torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)) * scale).to(dtype).cuda()


def layer(B, T, D, dtype, seed=1):
    td = TD[dtype]
    s = {n: rand(seed + i, B, T, D, dtype=td) for i, n in enumerate(("x", "decay", "gate", "z", "dy"))}
    s["taps"] = rand(seed + 5, D, W, dtype=td, scale=0.5)
    s["rate"] = torch.linspace(0.05, 1.0, D, device="cuda")
    s["weight"], s["bias"] = (1 + rand(seed + 6, D, scale=0.1)).to(td), rand(seed + 7, D, scale=0.1).to(td)
    return s


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kept", ["whole", "8 bits"])
@pytest.mark.parametrize("packed", [False, True])
def test_training(dtype, kept, packed):
    B, T, D = 2, 300, 192
    s = layer(B, T, D, dtype)
    seq = synth.segments(B, T, 60, 3, first=(1, 2)).cuda() if packed else None
    ids = None if seq is None else seq.cpu().numpy()
    c = dc.dynconv_fwd(s["x"], s["taps"], seq_idx=seq)
    kw = dict(gate=s["gate"], seq_idx=seq)
    h, chunks = dc.dynconv_scan_fwd(c, s["decay"], s["rate"], want_chunks=True, **kw)
    norm = dict(weight=s["weight"], bias=s["bias"], gate=s["z"])
    y = dc.dynconv_groupnorm_fwd(h, HEADS, **norm)
    n64 = {k: to64(v) for k, v in norm.items()}
    assert_close("h", h, scan_fwd(to64(c), to64(s["decay"]), to64(s["rate"]), to64(s["gate"]), ids)[0], h.dtype)
    assert_close("y", y, groupnorm_fwd(to64(h), HEADS, **n64), y.dtype)
    h64, c64, d64, g64 = to64(h), to64(c), to64(s["decay"]), to64(s["gate"])
    if kept == "whole":
        dh, dw, db, dz = dc.dynconv_groupnorm_bwd(h, HEADS, s["dy"], **norm)
        dcv, dd, dr, dg, _ = dc.dynconv_scan_bwd(c, s["decay"], s["rate"], dh, chunks=chunks, **kw)
    else:
        h64, c64, d64, g64 = (held8(v) for v in (h64, c64, d64, g64))
        p = [dc.dynconv_pack8(v) for v in (h, c, s["decay"], s["gate"])]
        dh, dw, db, dz = dc.dynconv_groupnorm_bwd(p[0], HEADS, s["dy"], **norm)
        dcv, dd, dr, dg, _ = dc.dynconv_scan_bwd(p[1], p[2], s["rate"], dh, gate=p[3], seq_idx=seq)
    ref = groupnorm_bwd(h64, HEADS, to64(s["dy"]), **n64)
    for name, got, r in zip(("dh", "dweight", "dbias", "dz"), (dh, dw, db, dz), ref):
        # a sum over 600 tokens in float32, 64 at a time: 128 roundings of 2^-24 of its magnitude at most
        assert_close(name, got, r, got.dtype, atol=1e-5 if name in ("dweight", "dbias") else None)
    ref = scan_bwd(c64, d64, to64(s["rate"]), g64, to64(dh), ids)
    for name, got, r in zip(("dc", "ddecay", "drate", "dgate"), (dcv, dd, dr, dg), ref):
        assert_close(name, got, r, got.dtype, atol=1e-5)
    dx, dtaps = dc.dynconv_bwd(s["x"], s["taps"], dcv, seq_idx=seq)
    rx, rt = conv_bwd(to64(s["x"]), to64(s["taps"]), to64(dcv), 1, ids)
    assert_close("dx", dx, rx, dx.dtype)
    assert_close("dtaps", dtaps, rt, dtaps.dtype, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_decoding_continues_a_prompt(dtype):
    """A prompt in one call, then token by token: the same rows as the whole sequence in one call."""
    B, T, T0, D = 3, 140, 131, 192
    s = layer(B, T, D, dtype, seed=20)
    c = dc.dynconv_fwd(s["x"], s["taps"])
    whole = dc.dynconv_scan_fwd(c, s["decay"], s["rate"], gate=s["gate"])
    cache = dc.dynconv_cache_fill(s["x"][:, :T0], W)
    state = dc.new_scan_state(B, D, "cuda")
    dc.dynconv_scan_fwd(c[:, :T0], s["decay"][:, :T0], s["rate"], gate=s["gate"][:, :T0], state=state, state_out=state)
    for t in range(T0, T):
        ct = dc.dynconv_decode_step(s["x"][:, t], s["taps"], cache, t)
        assert torch.equal(ct, c[:, t])
        ht = dc.dynconv_scan_step(ct, s["decay"][:, t], s["rate"], state, gate=s["gate"][:, t])
        # two roundings of the same value to the stored type: a step apart at most
        assert_close(f"h of token {t}", ht, to64(whole[:, t]), ht.dtype, rtol=2 * 2.0**-8 if dtype == "bf16" else 2 * 2.0**-11 if dtype == "f16" else 1e-5)
        yt = dc.dynconv_groupnorm_fwd(ht, HEADS, s["weight"], s["bias"], s["z"][:, t])
        ref = groupnorm_fwd(to64(ht)[:, None], HEADS, to64(s["weight"]), to64(s["bias"]), to64(s["z"])[:, t:t + 1])[:, 0]
        assert_close(f"y of token {t}", yt, ref, yt.dtype)
