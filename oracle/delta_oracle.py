"""Float64 NumPy reference of the gated delta rule and the gated RMS norm (tests and smoke() only).

The recurrence is written out token by token and its gradient walked back token by token
from the stored states; nothing is chunked and nothing is shared with the GPU path. Per
sequence and value head, with S [dk, dv]:

    P_t = e^{g_t} S_{t-1}        (zero at a document start, t > 0)
    w_t = v_t - P_t^T k_t,  u_t = beta_t w_t,  S_t = P_t + k_t u_t^T,  o_t = scale S_t^T q_t
"""
from __future__ import annotations

import numpy as np


def _unit(x, eps):
    """x over sqrt(|x|^2 + eps) along the last axis, and that length; x itself when eps is None."""
    if eps is None:
        return x, None
    length = np.sqrt(np.sum(x * x, axis=-1, keepdims=True) + eps)
    return x / length, length


def _starts(seq_idx, B, T):
    first = np.zeros((B, T), dtype=bool)
    if seq_idx is not None:
        seq_idx = np.asarray(seq_idx)
        first[:, 1:] = seq_idx[:, 1:] != seq_idx[:, :-1]
    return first


def delta_fwd(q, k, v, g, beta, scale, eps=None, seq_idx=None, state=None, keep=False):
    """(o [B,T,Hv,dv], final state [B,Hv,dk,dv]) of q, k [B,T,Hk,dk], v [B,T,Hv,dv], g, beta
    [B,T,Hv]; with keep also the P_t and S_t of every token."""
    q, k, v, g, beta = (np.asarray(a, dtype=np.float64) for a in (q, k, v, g, beta))
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2:]
    group = Hv // Hk
    q, _ = _unit(q, eps)
    k, _ = _unit(k, eps)
    first = _starts(seq_idx, B, T)
    o = np.zeros((B, T, Hv, dv))
    S = np.zeros((B, Hv, dk, dv)) if state is None else np.array(state, dtype=np.float64)
    past = []
    for t in range(T):
        kt, qt = np.repeat(k[:, t], group, axis=1), np.repeat(q[:, t], group, axis=1)  # [B,Hv,dk]
        a = np.where(first[:, t][:, None], 0.0, np.exp(g[:, t]))
        P = a[:, :, None, None] * S
        w = v[:, t] - np.sum(P * kt[..., None], axis=2)
        S = P + kt[..., None] * (beta[:, t][..., None] * w)[:, :, None, :]
        o[:, t] = scale * np.sum(S * qt[..., None], axis=2)
        if keep:
            past.append((P, w, S, a))
    return (o, S, past) if keep else (o, S)


def delta_bwd(q, k, v, g, beta, do, scale, eps=None, seq_idx=None, state=None, dstate_out=None):
    """(dq, dk, dv, dg, dbeta, dstate): gradients of <do, o> + <dstate_out, final state>."""
    q0, k0, v, g, beta, do = (np.asarray(a, dtype=np.float64) for a in (q, k, v, g, beta, do))
    B, T, Hk, dk = q0.shape
    Hv, dv = v.shape[2:]
    group = Hv // Hk
    past = delta_fwd(q0, k0, v, g, beta, scale, eps, seq_idx, state, keep=True)[2]
    q, ql = _unit(q0, eps)
    k, kl = _unit(k0, eps)
    dq, dkey = np.zeros((B, T, Hv, dk)), np.zeros((B, T, Hv, dk))
    dvv, dg, dbeta = np.zeros_like(v), np.zeros_like(g), np.zeros_like(beta)
    dS = np.zeros((B, Hv, dk, dv)) if dstate_out is None else np.array(dstate_out, dtype=np.float64)
    for t in reversed(range(T)):
        P, w, S, a = past.pop()
        kt, qt = np.repeat(k[:, t], group, axis=1), np.repeat(q[:, t], group, axis=1)
        dot = scale * do[:, t]  # [B,Hv,dv]
        dq[:, t] = np.sum(S * dot[:, :, None, :], axis=3)
        dS = dS + qt[..., None] * dot[:, :, None, :]
        du = np.sum(dS * kt[..., None], axis=2)
        bt = beta[:, t][..., None]
        dbeta[:, t] = np.sum(du * w, axis=-1)
        dw = bt * du
        dvv[:, t] = dw
        dkey[:, t] = np.sum(dS * (bt * w)[:, :, None, :], axis=3) - np.sum(P * dw[:, :, None, :], axis=3)
        dP = dS - kt[..., None] * dw[:, :, None, :]
        dg[:, t] = np.sum(dP * P, axis=(2, 3))
        dS = a[:, :, None, None] * dP
    if eps is not None:
        ql, kl = np.repeat(ql, group, axis=2), np.repeat(kl, group, axis=2)
        qr, kr = np.repeat(q, group, axis=2), np.repeat(k, group, axis=2)
        dq = (dq - qr * np.sum(qr * dq, axis=-1, keepdims=True)) / ql
        dkey = (dkey - kr * np.sum(kr * dkey, axis=-1, keepdims=True)) / kl
    dq, dkey = (x.reshape(B, T, Hk, group, dk).sum(axis=3) for x in (dq, dkey))
    return dq, dkey, dvv, dg, dbeta, dS


def _silu(z):
    s = 1.0 / (1.0 + np.exp(-z))
    return z * s, s * (1.0 + z * (1.0 - s))


def norm_fwd(x, weight=None, gate=None, eps=1e-6):
    """x / sqrt(mean(x^2) + eps) * weight * silu(gate) over the last axis."""
    x = np.asarray(x, dtype=np.float64)
    n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    y = n if weight is None else n * np.asarray(weight, dtype=np.float64)
    return y if gate is None else y * _silu(np.asarray(gate, dtype=np.float64))[0]


def norm_bwd(x, weight, gate, dy, eps=1e-6):
    """(dx, dweight, dgate) of <dy, norm_fwd(x, weight, gate)>; None where there is no input."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    D = x.shape[-1]
    length = np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    n = x / length
    w = np.ones(D) if weight is None else np.asarray(weight, dtype=np.float64)
    act, dact = (1.0, None) if gate is None else _silu(np.asarray(gate, dtype=np.float64))
    dn = dy * w * act
    dx = (dn - n * np.mean(dn * n, axis=-1, keepdims=True)) / length
    dw = None if weight is None else np.sum((dy * act * n).reshape(-1, D), axis=0)
    return dx, dw, None if gate is None else dy * n * w * dact
