"""Error bounds of the gated linear scan's kernels, element by element, in 64 bits.

With u = 2^-24: sigmoid(z) is good to (|z| + 5) u of itself (the rounded argument of the exponential, one ulp
each for it and the reciprocal, one sum), so for |z| up to 9 (what normal inputs reach) 14 u; g = rate s to 15 u,
a = e^-g to (15 g + 2) u and, as g e^-g < 0.37, to 8 u; 1 - a^2 to 20 u (below a half by its polynomial and
15 u of its argument; above, a^2's error over a difference of at least 0.39), b and 1/b to 12 u; an input
term b sg x to 30 u. A token's state goes through one map more per level (run, lane groups, wave, segment),
each a fused product and sum. All of it stays below C u per token of the sum of the absolute terms, C = 40, carried on by the
same recurrence.
"""
import numpy as np

from oracle import linear_scan, scan_terms
from oracle.delta_oracle import _starts

U = 2.0**-24
C = 40.0 * U


def fwd_bound(x, decay, rate, gate=None, seq_idx=None, state=None):
    """Bound of |h - exact| [B,T,D]."""
    _, a, _, _, u = scan_terms(x, decay, rate, gate)
    first = _starts(seq_idx, *u.shape[:2])
    size, _ = linear_scan(a, np.abs(u), first, None if state is None else np.abs(state))
    return linear_scan(a, C * size, first)[0]


def bwd_bounds(x, decay, rate, gate, dy, seq_idx=None, state=None, dstate_out=None):
    """Bounds of the errors of (dx, ddecay, drate, dgate, dstate), before any rounding of the result."""
    s, a, b, sg, u = scan_terms(x, decay, rate, gate)
    first = _starts(seq_idx, *u.shape[:2])
    ax = np.abs(np.asarray(x, dtype=np.float64))
    size, before = linear_scan(a, np.abs(u), first, None if state is None else np.abs(state))
    err, _ = linear_scan(a, C * size, first)
    err_before = np.concatenate([np.zeros_like(err[:, :1]), err[:, :-1]], 1)
    up, dsize = linear_scan(a, np.abs(np.asarray(dy, dtype=np.float64)), first,
                            None if dstate_out is None else np.abs(dstate_out), reverse=True)
    dh, dlast = linear_scan(a, C * up, first, reverse=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        slope = np.where(b > 0.0, a * a / b, 0.0)
    dx = b * sg * (dh + C * up)
    dgate = None if gate is None else dx * ax
    dl = s * (a * (dh * before + up * err_before) + dh * sg * ax * slope + C * up * (a * before + sg * ax * slope))
    return dx, rate * dl, dl.sum((0, 1)), dgate, dlast + C * dsize
