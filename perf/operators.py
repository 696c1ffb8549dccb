"""The gated delta rule and the gated RMS norm as workloads: cases, inputs, plain forms and exact values.

The layer that the short convolution feeds in a linear-attention model is, per value head,

    S_t = exp(g_t) S_{t-1} + k_t (beta_t (v_t - exp(g_t) S_{t-1}^T k_t))^T,    o_t = scale S_t^T q_t

(q and k of unit length when `qk_norm_eps` is given), followed by an RMS norm of o with a
weight and a SiLU gate; the block around it normalises the residual stream before and after
with the same norm. `own` selects who computes: False, the plain torch form below in 32
bits; True, the package's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
QK_EPS = 1e-6
NORM_EPS = 1e-5
CHUNK = 64


# ---------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------


def _delta(name, op, dtype, B, T, Hk, Hv, dk, dv, docs=0, state=False, norm=True):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "T": T, "Hk": Hk, "Hv": Hv, "dk": dk, "dv": dv,
            "docs": docs, "state": state, "norm": norm}


def _norm(name, dtype, rows, D, gate, res, train):
    return {"name": name, "op": "norm", "dtype": dtype, "rows": rows, "D": D, "gate": gate, "res": res, "train": train}


def listed():
    return [
        # one layer's training step at the convolution's headline shape (D = 2048 as 16 heads of 128)
        _delta("train_b8_t4096", "train", "bf16", 8, 4096, 16, 16, 128, 128),
        # packed documents, two value heads per key head, a length that ends inside a chunk
        _delta("train_packed_grouped", "train", "bf16", 2, 4001, 8, 16, 128, 128, docs=300),
        # a small model in float16, head sizes that fill no tile, continued from a carried state
        _delta("train_f16_odd_heads", "train", "f16", 3, 1000, 6, 6, 96, 80, state=True),
        # a float32 reference run, inputs normalised by the caller's own code
        _delta("train_f32", "train", "f32", 2, 777, 4, 8, 64, 64, norm=False),
        # a long prompt, its final state kept for decoding
        _delta("prefill_t32768", "prefill", "bf16", 1, 32768, 16, 16, 128, 128, state=True),
        # a short chat turn appended to a carried state: latency
        _delta("prefill_t70", "prefill", "bf16", 1, 70, 16, 32, 128, 128, state=True),
        # one decoding step of one sequence: latency
        _delta("step_b1", "step", "bf16", 1, 1, 16, 16, 128, 128),
        # one decoding step of a full serving batch, two value heads per key head
        _delta("step_b128_grouped", "step", "bf16", 128, 1, 16, 32, 128, 128),
        # the norm after the delta rule, per head, gated: training step
        _norm("norm_heads_gated", "bf16", 8 * 4096 * 16, 128, True, "none", True),
        # the norm before a block with the residual addition in it: training step
        _norm("norm_before_block", "bf16", 8 * 4096, 2048, False, "before", True),
        # the norm after a block, in float32 with an odd width: training step
        _norm("norm_after_block_f32", "f32", 5003, 1537, True, "after", True),
        # the norm before a block while decoding eight sequences: latency
        _norm("norm_before_block_step", "bf16", 8, 2048, False, "before", False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["train", "train", "prefill", "step", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    if kind == "norm":
        D = rng.choice([64, 128, 256, 512, 1024, 2048, 4096, _spread(rng, 3, 5000), _spread(rng, 3, 5000)])
        rows = _spread(rng, 1, max(1, min(300_000, 30_000_000 // D)))
        return {"op": "norm", "dtype": dtype, "rows": rows, "D": D, "gate": rng.random() < 0.5,
                "res": rng.choice(["none", "before", "after"]), "train": rng.random() < 0.6}
    group = rng.choice([1, 1, 2, 4])
    dk = rng.choice([128, 128, 64, _spread(rng, 8, 128)])
    dv = rng.choice([128, 128, 64, _spread(rng, 8, 256)])
    if kind == "step":
        Hk = rng.randint(1, 16)
        return {"op": "step", "dtype": dtype, "B": _spread(rng, 1, 128), "T": 1, "Hk": Hk, "Hv": Hk * min(group, 2),
                "dk": dk, "dv": dv, "docs": 0, "state": True, "norm": rng.random() < 0.8}
    B = _spread(rng, 1, 8)
    Hk = rng.randint(1, max(1, 16 // group))
    heads = B * Hk * group
    most = 4096 if kind == "train" else 32768
    T = _spread(rng, 1, max(2, min(most, (262_144 if kind == "train" else 524_288) // heads)))
    return {"op": kind, "dtype": dtype, "B": B, "T": T, "Hk": Hk, "Hv": Hk * group, "dk": dk, "dv": dv,
            "docs": rng.choice([0, 0, 20, 300]), "state": rng.random() < 0.5, "norm": rng.random() < 0.8}


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n = case["rows"] * case["D"]
        fwd = n * (2 + case["gate"] + (case["res"] != "none") + (case["res"] == "before"))  # x, gate, residual; y, h
        # the step reads dy, and the gradient of h, and writes dx, dgate and dresidual besides
        bwd = n * (2 + case["gate"] + (2 if case["res"] == "before" else 0)) if case["train"] else 0
        return {"bytes": (fwd + bwd) * e, "flops": n * (10 + (25 if case["train"] else 0))}
    B, T, Hk, Hv, dk, dv = (case[k] for k in ("B", "T", "Hk", "Hv", "dk", "dv"))
    act = B * T * (2 * Hk * dk + 2 * Hv * dv) * e + B * T * Hv * (4 + e)
    states = B * Hv * dk * dv * 4
    # the recurrence itself: S^T k, the rank-one update, S^T q (2 operations each per state element)
    flops = B * T * Hv * dk * dv * 6
    if case["op"] == "step":
        return {"bytes": act + 2 * states, "flops": flops}
    nbytes = act + states * ((1 if case["state"] else 0) + (1 if case["op"] == "prefill" else 0))
    if case["op"] == "train":
        # dO read, dq, dk, dv, dg, dbeta written; the recurrence backwards costs about twice its forward
        nbytes += act + states * (1 if case["state"] else 0)
        flops *= 3
    return {"bytes": nbytes, "flops": flops}


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
    if case["op"] == "norm":
        rows, D = case["rows"], case["D"]
        s["x"] = randn(rows, D).to(dt)
        s["weight"] = (1.0 + 0.1 * randn(D)).to(dt)
        s["gate"] = randn(rows, D).to(dt) if case["gate"] else None
        s["residual"] = (3.0 * randn(rows, D)).to(dt) if case["res"] != "none" else None
        s["alpha"] = 0.22 if case["res"] != "none" else 1.0  # the residual multiplier of depth-scaled models
        if case["train"]:
            s["dy"] = randn(rows, D).to(dt)
            s["dh"] = randn(rows, D).to(dt) if case["res"] == "before" else None
        return s
    B, T, Hk, Hv, dk, dv = (case[k] for k in ("B", "T", "Hk", "Hv", "dk", "dv"))
    # what the convolution and a SiLU leave: keys of one head lean the same way
    silu = torch.nn.functional.silu
    q, k, v = silu(1.5 * randn(B, T, Hk, dk)), silu(1.5 * randn(B, T, Hk, dk)), silu(1.5 * randn(B, T, Hv, dv))
    if not case["norm"]:
        q, k = (t * torch.rsqrt(t.square().sum(-1, keepdim=True) + QK_EPS) for t in (q, k))
    s["q"], s["k"], s["v"] = q.to(dt), k.to(dt), v.to(dt)
    s["beta"] = torch.sigmoid(randn(B, T, Hv)).to(dt)
    # the decay of a state-space layer: -A softplus(a + bias), A up to 16, steps of 0.001 to 0.1
    A = 1.0 + 15.0 * torch.rand(Hv, generator=gen, device=dev)
    step = torch.exp(torch.rand(Hv, generator=gen, device=dev) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    s["g"] = -A * torch.nn.functional.softplus(randn(B, T, Hv) + step + torch.log(-torch.expm1(-step)))
    s["seq"] = None
    if case["docs"]:
        starts = torch.rand(B, T, generator=gen, device=dev) < 1.0 / case["docs"]
        s["seq"] = starts.to(torch.int32).cumsum(1).to(torch.int32)
    has_state = case["state"] or case["op"] == "step"
    s["state"] = 0.3 * randn(B, Hv, dk, dv) if has_state else None
    s["do"] = randn(B, T, Hv, dv).to(dt) if case["op"] == "train" else None
    s["eps"] = QK_EPS if case["norm"] else None
    s["scale"] = dk ** -0.5
    if case["op"] == "step":
        for n in ("q", "k", "v", "g", "beta"):
            s[n] = s[n][:, 0].contiguous()
    return s


# ---------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------


def _bmm_t(a, b):
    return torch.matmul(a, b.transpose(-1, -2))


def _heads(t, group):
    """[B, T, H, d] -> [B * H * group, chunks, CHUNK, d] in float32, zeros behind the last token."""
    B, T, H, d = t.shape
    n = -(-T // CHUNK)
    out = torch.zeros(B, H, group, n * CHUNK, d, device=t.device)
    out[:, :, :, :T] = t.float().permute(0, 2, 1, 3).unsqueeze(2)
    return out.view(B * H * group, n, CHUNK, d)


def _unheads(t, B, T):
    N, n, C, d = t.shape
    return t.view(B, N // B, n * C, d)[:, :, :T].permute(0, 2, 1, 3)


class _Chunks:
    """What both directions share: the heads' chunks, their decays and the inverse of I + A."""

    def __init__(self, s):
        c = s["case"]
        B, T, Hv = c["B"], c["T"], c["Hv"]
        group = Hv // c["Hk"]
        self.B, self.T, self.group, self.scale, self.eps = B, T, group, s["scale"], s["eps"]
        self.q, self.k, self.v = _heads(s["q"], group), _heads(s["k"], group), _heads(s["v"], 1)
        self.rq = self.rk = None
        if self.eps is not None:
            self.rq = torch.rsqrt(self.q.square().sum(-1, keepdim=True) + self.eps)
            self.rk = torch.rsqrt(self.k.square().sum(-1, keepdim=True) + self.eps)
            self.q, self.k = self.q * self.rq, self.k * self.rk
        self.beta = _heads(s["beta"].unsqueeze(-1), 1)
        g = _heads(s["g"].unsqueeze(-1), 1).squeeze(-1)
        starts = torch.zeros_like(g)
        if s["seq"] is not None:
            first = torch.zeros(B, T, 1, 1, device=g.device)
            first[:, 1:, 0, 0] = (s["seq"][:, 1:] != s["seq"][:, :-1]).float()
            starts = _heads(first.expand(B, T, Hv, 1), 1).squeeze(-1)
        doc = starts.cumsum(-1)
        G = g.double().masked_fill(starts > 0, 0.0).cumsum(-1)  # differences of long sums: 64 bits
        low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=g.device).tril()
        seen = low & (doc.unsqueeze(-1) == doc.unsqueeze(-2))
        zero = torch.zeros((), dtype=torch.float64, device=g.device)
        self.decay = torch.where(seen, torch.exp(torch.where(seen, G.unsqueeze(-1) - G.unsqueeze(-2), zero)), zero).float()
        self.E = torch.where(doc == 0, torch.exp(G), zero).float().unsqueeze(-1)
        last = doc[..., -1:]
        self.D = torch.where(doc == last, torch.exp(G[..., -1:] - G), zero).float().unsqueeze(-1)
        self.gam = torch.where(last == 0, torch.exp(G[..., -1:]), zero).float().unsqueeze(-1)
        self.starts = starts
        self.M = (self.decay * _bmm_t(self.k, self.k)).tril(-1)
        A = self.beta * self.M
        inv = torch.eye(CHUNK, device=g.device).repeat(*A.shape[:2], 1, 1)
        for i in range(1, CHUNK):
            inv[:, :, i, :i] = -torch.matmul(A[:, :, i, None, :i], inv[:, :, :i, :i]).squeeze(-2)
        self.inv = inv
        self.P = self.scale * self.decay * _bmm_t(self.q, self.k)

    def states(self, s):
        """The state before each chunk, and the last one."""
        N, n = self.q.shape[:2]
        dk, dv = self.k.shape[-1], self.v.shape[-1]
        S = torch.zeros(N, dk, dv, device=self.q.device) if s["state"] is None else s["state"].float().reshape(N, dk, dv)
        before = []
        for c in range(n):
            before.append(S)
            k, u = self.k[:, c], None
            z = self.v[:, c] - self.E[:, c] * torch.matmul(k, S)
            u = torch.matmul(self.inv[:, c], self.beta[:, c] * z)
            S = self.gam[:, c] * S + torch.matmul((self.D[:, c] * k).transpose(-1, -2), u)
        return torch.stack(before, 1), S

    def forward(self, s):
        S0, last = self.states(s)
        self.S0 = S0
        self.KS = self.E * torch.matmul(self.k, S0)
        self.z = self.v - self.KS
        self.u = torch.matmul(self.inv, self.beta * self.z)
        self.QS = self.scale * self.E * torch.matmul(self.q, S0)
        return self.QS + torch.matmul(self.P, self.u), last

    def backward(self, s):
        do = _heads(s["do"], 1)
        n = do.shape[1]
        dS = torch.zeros_like(self.S0[:, 0])
        local = torch.matmul(self.P.transpose(-1, -2), do)
        after, dr = [None] * n, [None] * n
        for c in reversed(range(n)):
            after[c] = dS
            du = local[:, c] + self.D[:, c] * torch.matmul(self.k[:, c], dS)
            dr[c] = torch.matmul(self.inv[:, c].transpose(-1, -2), du)
            dS = (self.gam[:, c] * dS + torch.matmul((self.scale * self.E[:, c] * self.q[:, c]).transpose(-1, -2), do[:, c])
                  - torch.matmul((self.beta[:, c] * self.E[:, c] * self.k[:, c]).transpose(-1, -2), dr[c]))
        dS1, dr = torch.stack(after, 1), torch.stack(dr, 1)
        dz = self.beta * dr
        dP = self.decay * (self.scale * _bmm_t(do, self.u))
        dA = -_bmm_t(dr, self.u).tril(-1)
        dM = self.beta * dA * self.decay
        uS = self.D * _bmm_t(self.u, dS1)
        dq = self.scale * self.E * _bmm_t(do, self.S0) + torch.matmul(dP, self.k)
        dk = (torch.matmul(dP.transpose(-1, -2), self.q) + uS - self.E * _bmm_t(dz, self.S0)
              + torch.matmul(dM + dM.transpose(-1, -2), self.k))
        dbeta = (dr * self.z).sum(-1) + (dA * self.M).sum(-1)
        # the decay of token t scales every path from before t to t or later
        pair = (dP * _bmm_t(self.q, self.k) + dM * _bmm_t(self.k, self.k)).tril(-1)
        into = (do * self.QS).sum(-1) - (dz * self.KS).sum(-1)
        out = (self.k * uS).sum(-1)
        through = (self.gam * self.S0 * dS1).sum((-1, -2)).unsqueeze(-1)
        ahead = (pair.double().sum(-2) - pair.double().sum(-1) + out.double())
        dg = ((ahead.cumsum(-1) - ahead) + into.double().flip(-1).cumsum(-1).flip(-1) + through.double()).float()
        dg = dg.masked_fill(self.starts > 0, 0.0)
        if self.eps is not None:
            dq = self.rq * (dq - self.q * (self.q * dq).sum(-1, keepdim=True))
            dk = self.rk * (dk - self.k * (self.k * dk).sum(-1, keepdim=True))
        dq, dk = (t.view(self.B, -1, self.group, *t.shape[1:]).sum(2).view(-1, *t.shape[1:]) for t in (dq, dk))
        B, T, dt = self.B, self.T, s["q"].dtype
        out = [_unheads(dq, B, T).to(dt), _unheads(dk, B, T).to(dt), _unheads(dz, B, T).to(dt),
               _unheads(dg.unsqueeze(-1), B, T).squeeze(-1), _unheads(dbeta.unsqueeze(-1), B, T).squeeze(-1).to(dt)]
        return out + ([dS.view_as(s["state"])] if s["state"] is not None else [])


def _plain_step(s):
    group = s["v"].shape[1] // s["q"].shape[1]
    q, k = (t.float().repeat_interleave(group, 1) for t in (s["q"], s["k"]))
    if s["eps"] is not None:
        q, k = (t * torch.rsqrt(t.square().sum(-1, keepdim=True) + s["eps"]) for t in (q, k))
    S = s["state"].mul_(torch.exp(s["g"])[..., None, None])  # the cache is carried in place
    u = s["beta"].float().unsqueeze(-1) * (s["v"].float() - (S * k.unsqueeze(-1)).sum(-2))
    S.add_(k.unsqueeze(-1) * u.unsqueeze(-2))
    return [(s["scale"] * (S * q.unsqueeze(-1)).sum(-2)).to(s["q"].dtype), S]


def _plain_norm(s):
    res, alpha, dt = s["case"]["res"], s["alpha"], s["x"].dtype
    h = s["x"].float()
    out = []
    if res == "before":
        h = (s["residual"].float() + alpha * h).to(dt).float()  # the stored stream is what is normalised
        out.append(h.to(dt))
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + NORM_EPS)
    w = s["weight"].float()
    n = h * r
    act = torch.ones((), device=h.device)
    if s["gate"] is not None:
        z = s["gate"].float()
        sig = torch.sigmoid(z)
        act = z * sig
    y = n * w * act
    out.insert(0, ((s["residual"].float() + alpha * y) if res == "after" else y).to(dt))
    if not s["case"]["train"]:
        return out
    dy = s["dy"].float() * (alpha if res == "after" else 1.0)
    dn = dy * w * act
    dh = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    dw = (dy * act * n).sum(0)
    if res == "before":
        dh = dh + s["dh"].float()
        out += [(alpha * dh).to(dt), dh.to(dt)]
    else:
        out.append(dh.to(dt))
    out.append(dw)
    if s["gate"] is not None:
        out.append((dy * n * w * (sig * (1.0 + z * (1.0 - sig)))).to(dt))
    return out


# ---------------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------------


def _own(s):
    import dynamic_short_convolution_amd as dc

    c = s["case"]
    if c["op"] == "norm":
        kw = dict(gate=s["gate"], residual=s["residual"], residual_scale=s["alpha"],
                  residual_at="after" if c["res"] == "after" else "before", eps=NORM_EPS)
        got = dc.dynconv_norm_fwd(s["x"], s["weight"], **kw)
        y, h = got if c["res"] == "before" else (got, None)
        out = [y] + ([h] if h is not None else [])
        if not c["train"]:
            return out
        dx, dres, dw, dgate = dc.dynconv_norm_bwd(h if h is not None else s["x"], s["weight"], s["dy"], gate=s["gate"],
                                                  dh=s["dh"], residual_scale=s["alpha"],
                                                  residual_at=None if c["res"] == "none" else c["res"], eps=NORM_EPS)
        out += [dx] + ([dres] if c["res"] == "before" else []) + [dw]
        return out + ([dgate] if dgate is not None else [])
    kw = dict(scale=s["scale"], qk_norm_eps=s["eps"])
    args = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if c["op"] == "step":
        return [dc.dynconv_delta_step(*args, s["state"], **kw), s["state"]]
    kw.update(seq_idx=s["seq"], state=s["state"])
    if c["op"] == "prefill":
        return list(dc.dynconv_delta_fwd(*args, want_state=True, **kw))
    o = dc.dynconv_delta_fwd(*args, **kw)
    grads = dc.dynconv_delta_bwd(*args, s["do"], need_dstate=s["state"] is not None, **kw)
    return [o] + [t for t in grads if t is not None]


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "norm":
        return _plain_norm(state)
    if c["op"] == "step":
        return _plain_step(state)
    ch = _Chunks(state)
    o, last = ch.forward(state)
    o = _unheads(o, ch.B, ch.T).to(state["q"].dtype)
    if c["op"] == "prefill":
        return [o, last.view(c["B"], c["Hv"], c["dk"], c["dv"])]
    return [o] + ch.backward(state)


# ---------------------------------------------------------------------------------
# Exact values: the recurrence token by token, in 64 bits
# ---------------------------------------------------------------------------------


def _exact_norm(s):
    c, D = s["case"], s["case"]["D"]
    d = {n: None if s.get(n) is None else s[n].double() for n in ("x", "weight", "gate", "residual", "dy", "dh")}
    x, w, a = d["x"], d["weight"], s["alpha"]
    if c["res"] == "before":
        total = d["residual"] + a * x
        x = total.to(s["x"].dtype).double()  # what the storage type holds of it is what is normalised
    ms = (x * x).sum(-1, keepdim=True) / D + NORM_EPS
    act, dact = torch.ones_like(x), None
    if d["gate"] is not None:
        e = torch.exp(-d["gate"])
        act = d["gate"] / (1 + e)
        dact = 1 / (1 + e) + d["gate"] * e / (1 + e) ** 2
    y = x / ms.sqrt() * w * act
    out = [d["residual"] + a * y if c["res"] == "after" else y] + ([total] if c["res"] == "before" else [])
    if not c["train"]:
        return out
    dy = d["dy"] * (a if c["res"] == "after" else 1.0)
    up = dy * w * act
    dx = up / ms.sqrt() - x * (up * x).sum(-1, keepdim=True) / (D * ms ** 1.5)
    if c["res"] == "before":
        out += [a * (dx + d["dh"]), dx + d["dh"]]
    else:
        out += [dx]
    out += [(dy * act * x / ms.sqrt()).sum(0)]
    return out + ([dy * w * x / ms.sqrt() * dact] if dact is not None else [])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    B, T, Hk, Hv, dk, dv = (case[k] for k in ("B", "T", "Hk", "Hv", "dk", "dv"))
    if case["op"] == "step":
        for n in ("q", "k", "v", "g", "beta"):
            s[n] = s[n].unsqueeze(1)
    N, group, dev = B * Hv, Hv // Hk, s["q"].device
    if T * (N * dk * dv) * (12 if case["op"] == "train" else 4) > 5e12:  # over about 20 seconds
        return None

    def rows(t, rep):  # token-major, one row per value head
        return t.double().repeat_interleave(rep, 2).transpose(0, 1).reshape(T, N, *t.shape[3:]).contiguous()

    q0, k0, v = rows(s["q"], group), rows(s["k"], group), rows(s["v"], 1)
    beta, a = rows(s["beta"], 1), rows(s["g"], 1).exp()
    if s["seq"] is not None:
        new = torch.zeros(T, B, dtype=torch.bool, device=dev)
        new[1:] = (s["seq"][:, 1:] != s["seq"][:, :-1]).t()
        a = a.masked_fill(new.repeat_interleave(Hv, 1), 0.0)
    lq = lk = None
    q, k = q0, k0
    if s["eps"] is not None:
        lq, lk = ((t * t).sum(-1, keepdim=True).add(s["eps"]).sqrt() for t in (q0, k0))
        q, k = q0 / lq, k0 / lk
    S = torch.zeros(N, dk, dv, dtype=torch.float64, device=dev)
    if s["state"] is not None:
        S = s["state"].double().reshape(N, dk, dv).clone()

    def token(S, t):
        S = a[t].view(N, 1, 1) * S
        w = v[t] - torch.bmm(k[t].view(N, 1, dk), S).view(N, dv)
        return S, w

    seg, kept = 64, []
    o = torch.empty(T, N, dv, dtype=torch.float64, device=dev)
    for t in range(T):
        if t % seg == 0:
            kept.append(S)
        Sb, w = token(S, t)
        S = torch.baddbmm(Sb, k[t].view(N, dk, 1), (beta[t].view(N, 1) * w).view(N, 1, dv))
        o[t] = s["scale"] * torch.bmm(q[t].view(N, 1, dk), S).view(N, dv)

    def back(t, H):  # token-major to [B, T, H, ...]
        return t.view(T, B, H, *t.shape[2:]).transpose(0, 1)

    out = [back(o, Hv)]
    if case["op"] != "train":
        return ([out[0][:, 0]] if case["op"] == "step" else out) + [S.view(B, Hv, dk, dv)]
    do = rows(s["do"], 1) * s["scale"]
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    db, dg = torch.empty_like(beta), torch.empty_like(beta)
    dS = torch.zeros_like(S)
    for first in reversed(range(0, T, seg)):
        S, past = kept.pop(), []
        for t in range(first, min(T, first + seg)):
            Sb, w = token(S, t)
            S = torch.baddbmm(Sb, k[t].view(N, dk, 1), (beta[t].view(N, 1) * w).view(N, 1, dv))
            past.append((Sb, w, S))
        for t in reversed(range(first, min(T, first + seg))):
            Sb, w, S = past.pop()
            dq[t] = torch.bmm(S, do[t].view(N, dv, 1)).view(N, dk)
            dS = torch.baddbmm(dS, q[t].view(N, dk, 1), do[t].view(N, 1, dv))
            du = torch.bmm(k[t].view(N, 1, dk), dS).view(N, dv)
            u, dw = beta[t].view(N, 1) * w, beta[t].view(N, 1) * du
            db[t], dv_[t] = (du * w).sum(-1), dw
            dk_[t] = (torch.bmm(dS, u.view(N, dv, 1)) - torch.bmm(Sb, dw.view(N, dv, 1))).view(N, dk)
            dS = torch.baddbmm(dS, k[t].view(N, dk, 1), dw.view(N, 1, dv), alpha=-1.0)
            dg[t] = (dS * Sb).sum((1, 2))
            dS = a[t].view(N, 1, 1) * dS
    if s["eps"] is not None:
        dq = (dq - q * (q * dq).sum(-1, keepdim=True)) / lq
        dk_ = (dk_ - k * (k * dk_).sum(-1, keepdim=True)) / lk
    dq, dk_ = (back(t, Hv).reshape(B, T, Hk, group, dk).sum(3) for t in (dq, dk_))
    out += [dq, dk_, back(dv_, Hv), back(dg, Hv), back(db, Hv)]
    return out + ([dS.view(B, Hv, dk, dv)] if s["state"] is not None else [])
