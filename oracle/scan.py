"""fp64 reference of the gated linear recurrence and its backward pass (NumPy, one token
at a time).  Test infrastructure; shares no code with the HIP library.

    h_t = a_t h_{t-1} + b_t x_t,  y_t = h_t
    a = alpha or exp(alpha) (log);  b = beta, 1 - a (coupled) or 1
"""
from __future__ import annotations

import numpy as np


def _factors(alpha, beta, log, coupled):
    a = np.exp(alpha) if log else alpha
    b = beta if beta is not None else (1.0 - a if coupled else np.ones_like(a))
    return a, b


def _runs(T, B, offsets):
    """(batch row, sequence, first token, end) of every sequence."""
    if offsets is None:
        return [(b, b, 0, T) for b in range(B)]
    return [(0, i, int(p), int(q)) for i, (p, q) in enumerate(zip(offsets, offsets[1:]))]


def forward(x, alpha, beta=None, *, log=False, coupled=False, S0=None, offsets=None):
    """x, alpha, beta [B, T, D] fp64; S0 [B or n, D].  Returns y (rows of no sequence are NaN), ST."""
    B, T, D = x.shape
    n = B if offsets is None else len(offsets) - 1
    a, b = _factors(alpha, beta, log, coupled)
    S = np.zeros((n, D)) if S0 is None else np.array(S0, dtype=np.float64)
    y = np.full((B, T, D), np.nan)
    for row, i, p, q in _runs(T, B, offsets):
        for t in range(p, q):
            S[i] = a[row, t] * S[i] + b[row, t] * x[row, t]
            y[row, t] = S[i]
    return y, S


def backward(x, alpha, dy, beta=None, *, dST=None, log=False, coupled=False, S0=None, offsets=None):
    """Gradients of sum(y dy) + sum(ST dST): dx, dalpha (of alpha as given), dbeta or None, dS0."""
    B, T, D = x.shape
    n = B if offsets is None else len(offsets) - 1
    a, b = _factors(alpha, beta, log, coupled)
    y, _ = forward(x, alpha, beta, log=log, coupled=coupled, S0=S0, offsets=offsets)
    dx, da, db = (np.full((B, T, D), np.nan) for _ in range(3))
    dS = np.zeros((n, D)) if dST is None else np.array(dST, dtype=np.float64)
    for row, i, p, q in _runs(T, B, offsets):
        for t in reversed(range(p, q)):
            g = dS[i] + dy[row, t]
            before = y[row, t - 1] if t > p else (np.zeros(D) if S0 is None else S0[i])
            dx[row, t] = b[row, t] * g
            db[row, t] = g * x[row, t]
            da[row, t] = g * before - (g * x[row, t] if coupled else 0.0)
            dS[i] = a[row, t] * g
    return dx, da * a if log else da, None if beta is None else db, dS


def block_states(x, alpha, beta=None, *, block, **kw):
    """State after each block of `block` rows of a dense batch."""
    y, _ = forward(x, alpha, beta, **kw)
    T = x.shape[1]
    return y[:, [min(k + block, T) - 1 for k in range(0, T, block)]]
