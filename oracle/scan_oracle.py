"""Float64 NumPy reference of the gated linear scan, the group norm and activations in 8 bits (tests and
smoke() only).

The scan goes token by token and its gradient back token by token; the norm is written out over
its statistics' rows; nothing is chunked and nothing is shared with the GPU path.
"""
from __future__ import annotations

import numpy as np

from .delta_oracle import _silu, _starts


def _sigmoid(z):
    return 1.0 / (1.0 + np.exp(-np.asarray(z, dtype=np.float64)))


def scan_terms(x, decay, rate, gate=None):
    """(s, a, b, sg, u): sigmoid(decay), the decay, sqrt(1 - a^2), sigmoid(gate) and the input."""
    s = _sigmoid(decay)
    g = -np.asarray(rate, dtype=np.float64) * s
    b = np.sqrt(-np.expm1(2.0 * g))
    sg = np.ones_like(s) if gate is None else _sigmoid(gate)
    return s, np.exp(g), b, sg, b * sg * np.asarray(x, dtype=np.float64)


def linear_scan(a, u, first, state=None, reverse=False):
    """h_t = a_t h_{t-1} + u_t over axis 1 of [B,T,D] from `state`, 0 at `first` [B,T]; and the state
    that each token decays. reverse: h_t = u_t + a_{t+1} h_{t+1}, with the last token's from `state`."""
    B, T, D = u.shape
    h, before = np.zeros_like(u), np.zeros_like(u)
    prev = np.zeros((B, D)) if state is None else np.array(state, dtype=np.float64)
    for t in (reversed(range(T)) if reverse else range(T)):
        if reverse:
            h[:, t] = u[:, t] + prev
            prev = np.where(first[:, t, None], 0.0, a[:, t] * h[:, t])
        else:
            before[:, t] = np.where(first[:, t, None], 0.0, prev)
            prev = h[:, t] = a[:, t] * before[:, t] + u[:, t]
    return (h, prev) if reverse else (h, before)


def scan_fwd(x, decay, rate, gate=None, seq_idx=None, state=None):
    """(y [B,T,D], final state [B,D])."""
    _, a, _, _, u = scan_terms(x, decay, rate, gate)
    h, _ = linear_scan(a, u, _starts(seq_idx, *u.shape[:2]), state)
    final = h[:, -1] if h.shape[1] else (np.zeros((u.shape[0], u.shape[2])) if state is None else state)
    return h, final


def scan_bwd(x, decay, rate, gate, dy, seq_idx=None, state=None, dstate_out=None):
    """(dx, ddecay, drate, dgate, dstate): gradients of <dy, y> + <dstate_out, final state>."""
    s, a, b, sg, u = scan_terms(x, decay, rate, gate)
    first = _starts(seq_idx, *u.shape[:2])
    _, before = linear_scan(a, u, first, state)
    dh, dstate = linear_scan(a, np.asarray(dy, dtype=np.float64), first, dstate_out, reverse=True)
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        slope = np.where(b > 0.0, -a * a / b, 0.0)  # of sqrt(1 - e^{2g}) by g
    dg = dh * a * before + dh * sg * x * slope
    dgate = None if gate is None else dh * u * (1.0 - sg)
    return dh * b * sg, -dg * rate * s * (1.0 - s), np.sum(-dg * s, axis=(0, 1)), dgate, dstate


def pack8(x):
    """(codes, steps): integers and the power of two of every 64 channels; a group with a NaN or infinity
    has NaN steps."""
    x = np.asarray(x, dtype=np.float64)
    D = x.shape[-1]
    codes, steps = np.zeros(x.shape), np.zeros((*x.shape[:-1], -(-D // 64)))
    for i, lo in enumerate(range(0, D, 64)):
        part = x[..., lo:lo + 64]
        bad = ~np.isfinite(part).all(-1)
        part = np.where(bad[..., None], 0.0, part)
        e = np.maximum(np.frexp(np.abs(part).max(-1))[1] - 7, -126)
        step = np.exp2(e.astype(np.float64))
        codes[..., lo:lo + 64] = np.clip(np.rint(part / step[..., None]), -127, 127)
        steps[..., i] = np.where(bad, np.nan, step)
    return codes, steps


def held8(x):
    """The values that x has after 8 bits."""
    codes, steps = pack8(x)
    return codes * np.repeat(steps, 64, axis=-1)[..., :codes.shape[-1]]


def _rows(t, groups, over):
    """[n, C] as one row per statistic."""
    t = t.reshape(t.shape[0], groups, -1)
    return t if over == "token" else t.transpose(1, 0, 2).reshape(groups, -1)


def _back(r, n, groups, over):
    return r.reshape(n, -1) if over == "token" else r.reshape(groups, n, -1).transpose(1, 0, 2).reshape(n, -1)


def groupnorm_fwd(x, groups, weight=None, bias=None, gate=None, activation=None, over="token", lengths=None, eps=1e-5):
    """y [B,T,C] of act(n weight + bias) silu(gate), n normalised over a group's channels of a token or of
    all tokens of a sequence (the first lengths[b]; zeros behind them)."""
    x = np.asarray(x, dtype=np.float64)
    y = np.zeros_like(x)
    for b in range(x.shape[0]):
        n = x.shape[1] if lengths is None else int(np.clip(lengths[b], 0, x.shape[1]))
        if n == 0:
            continue
        r = _rows(x[b, :n], groups, over)
        r = r - r.mean(-1, keepdims=True)
        z = _back(r / np.sqrt((r * r).mean(-1, keepdims=True) + eps), n, groups, over)
        z = z * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
        if activation == "silu":
            z = _silu(z)[0]
        y[b, :n] = z if gate is None else z * _silu(np.asarray(gate, dtype=np.float64)[b, :n])[0]
    return y


def groupnorm_bwd(x, groups, dy, weight=None, bias=None, gate=None, activation=None, over="token", lengths=None, eps=1e-5):
    """(dx, dweight, dbias, dgate) of <dy, groupnorm_fwd(...)>; dgate None without a gate."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    C = x.shape[2]
    w = np.ones(C) if weight is None else np.asarray(weight, dtype=np.float64)
    dx, dgate = np.zeros_like(x), None if gate is None else np.zeros_like(x)
    dw, db = np.zeros(C), np.zeros(C)
    for b in range(x.shape[0]):
        n = x.shape[1] if lengths is None else int(np.clip(lengths[b], 0, x.shape[1]))
        if n == 0:
            continue
        r = _rows(x[b, :n], groups, over)
        r = r - r.mean(-1, keepdims=True)
        std = np.sqrt((r * r).mean(-1, keepdims=True) + eps)
        r = r / std
        norm = _back(r, n, groups, over)
        z = norm * w + (0.0 if bias is None else bias)
        act, slope = _silu(z) if activation == "silu" else (z, np.ones_like(z))
        up = dy[b, :n]
        if gate is not None:
            opened, dopen = _silu(np.asarray(gate, dtype=np.float64)[b, :n])
            dgate[b, :n] = up * act * dopen
            up = up * opened
        dz = up * slope
        dw += (dz * norm).sum(0)
        db += dz.sum(0)
        dn = _rows(dz * w, groups, over)
        dx[b, :n] = _back((dn - dn.mean(-1, keepdims=True) - r * (dn * r).mean(-1, keepdims=True)) / std, n, groups, over)
    return dx, dw, db, dgate
