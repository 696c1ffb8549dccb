"""The gated linear scan, the group norm and 8-bit checkpoints as workloads: cases, inputs, plain forms, exact values.

What a linear-recurrent layer puts behind its short convolution. Per channel,

    a_t = exp(-rate sigmoid(decay_t)),    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(gate_t) x_t,

then a group norm of h (per token or over a whole sequence) with weight, bias, SiLU and a SiLU gate. For training, what
the backward passes read of the forward's inputs may be held in 8 bits: integers of at most 127 times a power of two
that each 64 channels of a token share. `own` selects who computes: False, the plain torch form below in 32 bits; True,
the package's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NORM_EPS = 1e-5
PACK = 64  # channels of a token that share a scale


# ---------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------


def _scan(name, op, dtype, B, T, D, docs=0, state=False, gate=True, ckpt=False):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "T": T, "D": D, "docs": docs, "state": state, "gate": gate,
            "ckpt": ckpt}


def _group(name, dtype, B, T, groups, width, over, gate, silu, train, lengths=False, ckpt=False):
    return {"name": name, "op": "group", "dtype": dtype, "B": B, "T": T, "groups": groups, "width": width, "over": over,
            "gate": gate, "silu": silu, "train": train, "lengths": lengths, "ckpt": ckpt}


def listed():
    return [
        # one layer's training step at the convolution's headline shape
        _scan("scan_train_b8_t4096", "scan_train", "bf16", 8, 4096, 2048),
        # packed documents in float16, continued from a carried state, a width that fills no block of 64 channels
        _scan("scan_train_f16_packed", "scan_train", "f16", 3, 1501, 1000, docs=200, state=True),
        # a float32 reference run of a small odd model, no input gate
        _scan("scan_train_f32", "scan_train", "f32", 2, 777, 515, gate=False),
        # the headline training step with the forward's inputs kept in 8 bits
        _scan("scan_train_checkpoints", "scan_train", "bf16", 8, 4096, 2048, ckpt=True),
        # a long prompt of one sequence, its final state kept for decoding
        _scan("scan_prefill_t32768", "scan_prefill", "bf16", 1, 32768, 2048, state=True),
        # a short chat turn appended to a carried state: latency
        _scan("scan_prefill_t70", "scan_prefill", "bf16", 1, 70, 2048, state=True),
        # one decoding step of eight sequences: latency
        _scan("scan_step_b8", "scan_step", "bf16", 8, 1, 2048, state=True),
        # the norm behind the recurrence, 16 heads of 128 channels, gated: training step
        _group("group_tokens_gated", "bf16", 8, 4096, 16, 128, "token", True, False, True),
        # odd groups in float32 with the activation: training step
        _group("group_tokens_f32", "f32", 1, 5003, 27, 57, "token", False, True, True),
        # the norm behind a convolution stack, over the tokens of padded sequences: training step
        _group("group_sequences", "bf16", 8, 4096, 32, 64, "sequence", False, True, True, lengths=True),
        # the gated norm while decoding eight sequences: latency
        _group("group_tokens_step", "bf16", 8, 1, 16, 128, "token", True, False, False),
        # a block's float32 residual stream kept in 8 bits and read back, an odd width
        {"name": "checkpoint_f32", "op": "pack", "dtype": "f32", "rows": 5003, "D": 1537},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["scan_train", "scan_train", "scan_prefill", "scan_step", "group", "group", "group", "pack"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    most = 30_000_000 if dtype == "f32" else 60_000_000
    if kind == "pack":
        D = rng.choice([64, 128, 256, 2048, 4096, _spread(rng, 1, 6000)])
        return {"op": "pack", "dtype": dtype, "rows": _spread(rng, 1, min(300_000, most // D)), "D": D}
    B = _spread(rng, 1, 8)
    if kind == "group":
        width = rng.choice([32, 64, 64, 128, 256, _spread(rng, 16, 2048)])
        groups = _spread(rng, 1, max(2, min(64, 8192 // width)))
        T = _spread(rng, 1, min(32768, most // (B * width * groups)))
        over = rng.choice(["token", "token", "sequence"])
        train = rng.random() < 0.7
        return {"op": "group", "dtype": dtype, "B": B, "T": T, "groups": groups, "width": width, "over": over,
                "gate": rng.random() < 0.5, "silu": rng.random() < 0.5, "train": train,
                "lengths": over == "sequence" and rng.random() < 0.5, "ckpt": train and rng.random() < 0.3}
    D = rng.choice([256, 512, 1024, 2048, 4096, _spread(rng, 1, 5000), _spread(rng, 1, 5000)])
    if kind == "scan_step":
        return {"op": kind, "dtype": dtype, "B": _spread(rng, 1, 512), "T": 1, "D": D, "docs": 0, "state": True,
                "gate": rng.random() < 0.8, "ckpt": False}
    return {"op": kind, "dtype": dtype, "B": B, "T": _spread(rng, 1, min(32768, most // (B * D))), "D": D,
            "docs": rng.choice([0, 0, 20, 300]), "state": rng.random() < 0.5, "gate": rng.random() < 0.8,
            "ckpt": kind == "scan_train" and rng.random() < 0.3}


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "pack":
        n = case["rows"] * case["D"]
        return {"bytes": 2 * n * e, "flops": 4 * n}
    if case["op"] == "group":
        n = case["B"] * case["T"] * case["groups"] * case["width"]
        # x, gate, y; the step reads dy and writes dx and dgate besides
        tensors = 2 + case["gate"] + ((2 + case["gate"]) if case["train"] else 0)
        return {"bytes": n * e * tensors, "flops": n * (12 + (25 if case["train"] else 0))}
    n, states = case["B"] * case["T"] * case["D"], case["B"] * case["D"] * 4
    # x, decay, gate, y; the step reads dy and writes dx, ddecay and dgate besides
    tensors = 3 + case["gate"] + ((3 + case["gate"]) if case["op"] == "scan_train" else 0)
    carried = states * (1 if case["state"] else 0) + states * (1 if case["op"] != "scan_train" or case["state"] else 0)
    return {"bytes": n * e * tensors + carried, "flops": n * (20 + (40 if case["op"] == "scan_train" else 0))}


# ---------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    s = {"case": case}
    if case["op"] == "pack":
        s["x"] = (randn(case["rows"], case["D"]) * torch.exp(randn(case["rows"], 1))).to(dt)
        return s
    if case["op"] == "group":
        B, T, C = case["B"], case["T"], case["groups"] * case["width"]
        s["x"] = (randn(B, T, C) + 0.5 * randn(C)).to(dt)
        s["weight"], s["bias"] = (1.0 + 0.1 * randn(C)).to(dt), (0.1 * randn(C)).to(dt)
        s["gate"] = randn(B, T, C).to(dt) if case["gate"] else None
        s["dy"] = randn(B, T, C).to(dt) if case["train"] else None
        s["lengths"] = None
        if case["lengths"]:
            s["lengths"] = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        return s
    B, T, D = case["B"], case["T"], case["D"]
    s["x"], s["decay"] = randn(B, T, D).to(dt), randn(B, T, D).to(dt)
    s["gate"] = randn(B, T, D).to(dt) if case["gate"] else None
    # decays of 0.9 to 0.999 a token at an open decay gate's eighth: memories of ten to a thousand tokens
    s["rate"] = -8.0 * torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device=dev))
    s["seq"] = None
    if case["docs"]:
        first = torch.rand(B, T, generator=gen, device=dev) < 1.0 / case["docs"]
        s["seq"] = first.to(torch.int32).cumsum(1).to(torch.int32)
    s["state"] = 0.5 * randn(B, D) if case["state"] else None
    s["dy"] = randn(B, T, D).to(dt) if case["op"] == "scan_train" else None
    if case["op"] == "scan_step":
        for n in ("x", "decay", "gate"):
            s[n] = None if s[n] is None else s[n][:, 0].contiguous()
    return s


# ---------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------


def _held(t):
    """The values that t has after 8 bits, in float32."""
    D = t.shape[-1]
    v = torch.nn.functional.pad(t.float(), (0, -D % PACK)).unflatten(-1, (-1, PACK))
    exponent = (torch.frexp(v.abs().amax(-1, keepdim=True)).exponent - 7).clamp_min(-126)
    codes = torch.ldexp(v, -exponent).round().clamp(-127, 127)
    return torch.ldexp(codes, exponent).flatten(-2)[..., :D]


def _prefix(a, u, reverse=False):
    """h_t = a_t h_{t-1} + u_t along dimension 1 from h = 0 (reverse: from h_{t+1}), by doubling."""
    if reverse:
        return _prefix(a.flip(1), u.flip(1)).flip(1)
    step = 1
    while step < u.shape[1]:
        u = torch.cat([u[:, :step], u[:, step:] + a[:, step:] * u[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return u


def _gates(x, decay, gate, rate):
    """sigmoid(decay), a, sqrt(1 - a^2), sigmoid(gate) and the input u, in float32."""
    sd = torch.sigmoid(decay.float())
    g = -rate * sd
    b = torch.sqrt(-torch.expm1(2.0 * g))
    sg = torch.sigmoid(gate.float()) if gate is not None else torch.ones((), device=x.device)
    return sd, torch.exp(g), b, sg, b * sg * x.float()


def _starts(seq):
    first = torch.zeros(seq.shape, dtype=torch.bool, device=seq.device)
    first[:, 1:] = seq[:, 1:] != seq[:, :-1]
    return first.unsqueeze(-1)


def _plain_states(s, a, u):
    if s["seq"] is not None:
        a = a.masked_fill(_starts(s["seq"]), 0.0)
    if s["state"] is not None:
        u = torch.cat([u[:, :1] + a[:, :1] * s["state"].unsqueeze(1), u[:, 1:]], 1)
    return a, _prefix(a, u)


def _plain_scan(s):
    c, dt = s["case"], s["x"].dtype
    if c["op"] == "scan_step":
        _, a, _, _, u = _gates(s["x"], s["decay"], s["gate"], s["rate"])
        h = s["state"].mul_(a).add_(u)  # the state is carried in place
        return [h.to(dt), h]
    sd, a, b, sg, u = _gates(s["x"], s["decay"], s["gate"], s["rate"])
    through, h = _plain_states(s, a, u)
    out = [h.to(dt)]
    if c["op"] == "scan_prefill":
        return out + [h[:, -1]]
    x = s["x"].float()
    if c["ckpt"]:
        x, decay, gate = _held(s["x"]), _held(s["decay"]), None if s["gate"] is None else _held(s["gate"])
        sd, a, b, sg, u = _gates(x, decay, gate, s["rate"])
        through, h = _plain_states(s, a, u)
    before = torch.zeros_like(h[:, :1]) if s["state"] is None else s["state"].unsqueeze(1)
    before = torch.cat([before, h[:, :-1]], 1)
    if s["seq"] is not None:
        before = before.masked_fill(_starts(s["seq"]), 0.0)
    # dh_t = dy_t + a_{t+1} dh_{t+1}
    dh = _prefix(torch.cat([through[:, 1:], torch.zeros_like(through[:, :1])], 1), s["dy"].float(), reverse=True)
    dg = a * dh * before - torch.where(b > 0, a * a / b, torch.zeros((), device=b.device)) * dh * sg * x
    out += [(dh * b * sg).to(dt), (dg * (-s["rate"] * sd * (1.0 - sd))).to(dt), -(dg * sd).sum((0, 1), dtype=torch.float64).float()]
    if s["gate"] is not None:
        out.append((dh * u * (1.0 - sg)).to(dt))
    if s["state"] is not None:
        out.append(through[:, 0] * dh[:, 0])
    return out


def _plain_group(s):
    c, dt = s["case"], s["x"].dtype
    B, T, G, width = c["B"], c["T"], c["groups"], c["width"]
    dims = (-1,) if c["over"] == "token" else (1, -1)
    keep = torch.ones((), device=s["x"].device)
    count = torch.full((B, 1, 1, 1), float(width * (T if c["over"] == "sequence" else 1)), device=s["x"].device)
    if s["lengths"] is not None:
        keep = (torch.arange(T, device=s["x"].device) < s["lengths"].unsqueeze(1)).float().view(B, T, 1, 1)
        count = (s["lengths"].float() * width).clamp_min(1.0).view(B, 1, 1, 1)

    def split(t):
        return t.float().view(B, T, G, width)

    def mean(t):  # long sums in 64 bits
        return ((t * keep).sum(dims, keepdim=True, dtype=torch.float64) / count).float()

    def norm(x):
        x = x - mean(x)
        rstd = torch.rsqrt(mean(x * x) + NORM_EPS)
        return x * rstd, rstd

    w, b = (s[n].float().view(G, width) for n in ("weight", "bias"))
    n, rstd = norm(split(s["x"]))
    act = torch.sigmoid(split(s["gate"])) * split(s["gate"]) if c["gate"] else torch.ones((), device=n.device)
    z = n * w + b
    y = (z * torch.sigmoid(z) if c["silu"] else z) * act * keep
    out = [y.to(dt).view(B, T, G * width)]
    if not c["train"]:
        return out
    if c["ckpt"]:
        n, rstd = norm(split(_held(s["x"])))
        z = n * w + b
    sz = torch.sigmoid(z)
    dy = split(s["dy"]) * keep
    dz = dy * act * ((sz * (1.0 + z * (1.0 - sz))) if c["silu"] else 1.0)
    dn = dz * w
    dx = rstd * (dn - mean(dn) - n * mean(dn * n)) * keep
    out += [dx.to(dt).view(B, T, G * width), (dz * n).sum((0, 1), dtype=torch.float64).float().view(-1),
            dz.sum((0, 1), dtype=torch.float64).float().view(-1)]
    if c["gate"]:
        g = split(s["gate"])
        sg = torch.sigmoid(g)
        out.append((dy * (z * sz if c["silu"] else z) * sg * (1.0 + g * (1.0 - sg))).to(dt).view(B, T, G * width))
    return out


# ---------------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------------


def _own(s):
    import dynamic_short_convolution_amd as dc

    c = s["case"]
    if c["op"] == "pack":
        return [dc.dynconv_unpack8(dc.dynconv_pack8(s["x"]), s["x"].dtype)]
    if c["op"] == "group":
        kw = dict(weight=s["weight"], bias=s["bias"], gate=s["gate"], activation="silu" if c["silu"] else None,
                  over=c["over"], lengths=s["lengths"], eps=NORM_EPS)
        if not c["train"]:
            return [dc.dynconv_groupnorm_fwd(s["x"], c["groups"], **kw)]
        y, stats = dc.dynconv_groupnorm_fwd(s["x"], c["groups"], want_stats=True, **kw)
        if c["ckpt"]:
            grads = dc.dynconv_groupnorm_bwd(dc.dynconv_pack8(s["x"]), c["groups"], s["dy"], **kw)
        else:
            grads = dc.dynconv_groupnorm_bwd(s["x"], c["groups"], s["dy"], stats=stats, **kw)
        return [y] + [t for t in grads if t is not None]
    if c["op"] == "scan_step":
        return [dc.dynconv_scan_step(s["x"], s["decay"], s["rate"], s["state"], gate=s["gate"]), s["state"]]
    kw = dict(gate=s["gate"], seq_idx=s["seq"], state=s["state"])
    if c["op"] == "scan_prefill":
        return list(dc.dynconv_scan_fwd(s["x"], s["decay"], s["rate"], want_state=True, **kw))
    if c["ckpt"]:
        y = dc.dynconv_scan_fwd(s["x"], s["decay"], s["rate"], **kw)
        x, decay = dc.dynconv_pack8(s["x"]), dc.dynconv_pack8(s["decay"])
        kw["gate"] = None if s["gate"] is None else dc.dynconv_pack8(s["gate"])
        grads = dc.dynconv_scan_bwd(x, decay, s["rate"], s["dy"], need_dstate=s["state"] is not None, **kw)
    else:
        y, chunks = dc.dynconv_scan_fwd(s["x"], s["decay"], s["rate"], want_chunks=True, **kw)
        grads = dc.dynconv_scan_bwd(s["x"], s["decay"], s["rate"], s["dy"], chunks=chunks,
                                    need_dstate=s["state"] is not None, **kw)
    return [y] + [t for t in grads if t is not None]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "pack":
        return [_held(state["x"]).to(state["x"].dtype)]
    return _plain_group(state) if op == "group" else _plain_scan(state)


# ---------------------------------------------------------------------------------
# Exact values: the definitions in 64 bits
# ---------------------------------------------------------------------------------


def _exact_held(t):
    v, D = t.double(), t.shape[-1]
    out = torch.empty_like(v)
    for lo in range(0, D, PACK):
        part = v[..., lo:lo + PACK]
        top = part.abs().amax(-1, keepdim=True)
        # the power of two at or below the largest value, 64 steps of it
        step = torch.exp2(torch.floor(torch.log2(top.clamp_min(2.0 ** -120))) - 6.0)
        step = torch.where(step * 64.0 > top.clamp_min(2.0 ** -120), step / 2.0, step)
        step = torch.where(step * 128.0 <= top, step * 2.0, step)
        out[..., lo:lo + PACK] = (part / step).round().clamp(-127.0, 127.0) * step
    return out


def _exact_scan(s):
    c = s["case"]
    one = c["op"] == "scan_step"
    names = ("x", "decay", "gate")

    def forward(v):
        x, decay, gate = v
        sd = 1.0 / (1.0 + torch.exp(-decay))
        sg = 1.0 / (1.0 + torch.exp(-gate)) if gate is not None else torch.ones_like(x)
        g = -s["rate"].double() * sd
        a, b = torch.exp(g), torch.sqrt(-torch.expm1(2.0 * g))
        B, T, D = x.shape
        h = torch.empty_like(x)
        prev = torch.zeros(B, D, dtype=torch.float64, device=x.device) if s["state"] is None else s["state"].double().clone()
        kept = torch.empty_like(x)  # the state that each token decays
        for t in range(T):
            if new is not None and t > 0:
                prev = prev * new[:, t:t + 1]
            kept[:, t] = prev
            prev = torch.addcmul(b[:, t] * sg[:, t] * x[:, t], a[:, t], prev)
            h[:, t] = prev
        return sd, sg, g, a, b, kept, h

    new = None  # 0 at the first token of a document, 1 elsewhere
    if s["seq"] is not None:
        new = torch.ones_like(s["seq"], dtype=torch.float64)
        new[:, 1:] = (s["seq"][:, 1:] == s["seq"][:, :-1]).double()
    v = [None if s[n] is None else (s[n].unsqueeze(1) if one else s[n]).double() for n in names]
    sd, sg, g, a, b, kept, h = forward(v)
    if one:
        return [h[:, 0], h[:, 0]]
    if c["op"] == "scan_prefill":
        return [h, h[:, -1]]
    y = h
    if c["ckpt"]:
        v = [None if s[n] is None else _exact_held(s[n]) for n in names]
        sd, sg, g, a, b, kept, h = forward(v)
    dy, x = s["dy"].double(), v[0]
    dh = torch.empty_like(dy)
    back = torch.zeros_like(dy[:, 0])
    for t in reversed(range(dy.shape[1])):
        dh[:, t] = dy[:, t] + back
        back = a[:, t] * dh[:, t]
        if new is not None and t > 0:
            back = back * new[:, t:t + 1]
    db = dh * sg * x
    # sqrt(1 - e^{2g}) by g; 0 where the channel neither forgets nor takes in
    dg = dh * kept * a + db * torch.where(b > 0, -(a * a) / b, torch.zeros_like(b))
    out = [y, dh * b * sg, dg * g * (1.0 - sd), (-dg * sd).sum((0, 1))]
    if s["gate"] is not None:
        out.append(dh * b * x * sg * (1.0 - sg))
    return out + ([back] if s["state"] is not None else [])


def _exact_group(s):
    c = s["case"]
    B, T, G, width = c["B"], c["T"], c["groups"], c["width"]
    lengths = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    w, b = s["weight"].double(), s["bias"].double()
    zeros = torch.zeros(B, T, G * width, dtype=torch.float64, device=w.device)
    y, dx, dgate = zeros, zeros.clone() if c["train"] else None, zeros.clone() if c["train"] and c["gate"] else None
    dw, db = torch.zeros_like(w), torch.zeros_like(b)

    def normed(x):  # rows of one statistic each
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        return (x - mean) / torch.sqrt(var + NORM_EPS), torch.sqrt(var + NORM_EPS)

    def rows(t):  # [tokens, C] to one row per statistic, and back
        t = t.view(-1, G, width)
        return t if c["over"] == "token" else t.transpose(0, 1).reshape(G, -1)

    def tokens(t, n):
        return t.reshape(n, -1) if c["over"] == "token" else t.view(G, n, width).transpose(0, 1).reshape(n, -1)

    for i, n in enumerate(lengths):
        if n == 0:
            continue
        z = tokens(normed(rows(s["x"][i, :n].double()))[0], n) * w + b
        gate = s["gate"][i, :n].double() if c["gate"] else None
        open_ = gate / (1.0 + torch.exp(-gate)) if c["gate"] else torch.ones_like(z)
        y[i, :n] = (z / (1.0 + torch.exp(-z)) if c["silu"] else z) * open_
        if not c["train"]:
            continue
        xh = _exact_held(s["x"][i, :n]) if c["ckpt"] else s["x"][i, :n].double()
        nr, std = normed(rows(xh))
        nt = tokens(nr, n)
        z = nt * w + b
        e = torch.exp(-z)
        dz = s["dy"][i, :n].double() * open_ * ((1.0 + e + z * e) / (1.0 + e) ** 2 if c["silu"] else 1.0)
        dw += (dz * nt).sum(0)
        db += dz.sum(0)
        up = rows(dz * w)
        dx[i, :n] = tokens((up - up.mean(-1, keepdim=True) - nr * (up * nr).mean(-1, keepdim=True)) / std, n)
        if c["gate"]:
            eg = torch.exp(-gate)
            dgate[i, :n] = (s["dy"][i, :n].double() * (z / (1.0 + e) if c["silu"] else z)
                            * (1.0 + eg + gate * eg) / (1.0 + eg) ** 2)
    return [y] + ([dx, dw, db] if c["train"] else []) + ([dgate] if dgate is not None else [])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pack":
        return [_exact_held(s["x"])]
    return _exact_group(s) if case["op"] == "group" else _exact_scan(s)
