"""fp64 reference of the trainable delta rule (gdr_delta_fwd, gdr_delta_bwd, gdr_delta_step), token by token.

    X = a S_{t-1},  e = v - X^T k,  S_t = X + k (beta e)^T,  o = S_t^T q,   a = exp(log_gate)

q, k [T, Hk, dk], v [T, Hv, dv], log_gate, beta [T, Hv], S [Hv, dk, dv]; value head h goes with key head
h // (Hv // Hk).  One sequence a call."""
from __future__ import annotations

import numpy as np


def _heads(x, Hv):
    return np.repeat(x, Hv // x.shape[1], axis=1)


def forward(q, k, v, log_gate, beta, S0=None):
    """(o [T, Hv, dv], ST, the states after each token [T, Hv, dk, dv])."""
    T, Hv, dv = v.shape
    q, k = _heads(q, Hv), _heads(k, Hv)
    S = np.zeros((Hv, q.shape[-1], dv)) if S0 is None else S0.astype(np.float64)
    o, states = np.empty((T, Hv, dv)), np.empty((T,) + S.shape)
    for t in range(T):
        X = np.exp(log_gate[t])[:, None, None] * S
        e = v[t] - np.einsum("hij,hi->hj", X, k[t])
        S = X + k[t][:, :, None] * (beta[t][:, None] * e)[:, None, :]
        o[t] = np.einsum("hij,hi->hj", S, q[t])
        states[t] = S
    return o, S, states


def backward(q, k, v, log_gate, beta, d_o, dST=None, S0=None):
    """Gradients of q, k, v, log_gate, beta and S0: the chain rule, token by token from the end.  Then the sizes of the
    dot products that those of log_gate and beta are: the product of their factors' norms, which rounding errors go with."""
    T, Hv, dv = v.shape
    Hk, dk = q.shape[1:]
    states = forward(q, k, v, log_gate, beta, S0)[2]
    qh, kh = _heads(q, Hv), _heads(k, Hv)
    G = np.zeros((Hv, dk, dv)) if dST is None else dST.astype(np.float64)
    gq, gk, gv = np.zeros((T, Hv, dk)), np.zeros((T, Hv, dk)), np.zeros((T, Hv, dv))
    gg, gb, size_g, size_b = (np.zeros((T, Hv)) for _ in range(4))
    for t in reversed(range(T)):
        before = states[t - 1] if t else (np.zeros((Hv, dk, dv)) if S0 is None else S0.astype(np.float64))
        X = np.exp(log_gate[t])[:, None, None] * before
        e = v[t] - np.einsum("hij,hi->hj", X, kh[t])
        gq[t] = np.einsum("hij,hj->hi", states[t], d_o[t])
        G = G + qh[t][:, :, None] * d_o[t][:, None, :]
        d = np.einsum("hij,hi->hj", G, kh[t])          # of beta e
        gb[t] = (d * e).sum(-1)
        size_b[t] = np.linalg.norm(d, axis=-1) * np.linalg.norm(e, axis=-1)
        de = beta[t][:, None] * d
        gv[t] = de
        gk[t] = np.einsum("hij,hj->hi", G, beta[t][:, None] * e) - np.einsum("hij,hj->hi", X, de)
        dX = G - kh[t][:, :, None] * de[:, None, :]
        gg[t] = (dX * X).sum((-2, -1))
        size_g[t] = np.linalg.norm(dX, axis=(-2, -1)) * np.linalg.norm(X, axis=(-2, -1))
        G = np.exp(log_gate[t])[:, None, None] * dX
    share = lambda x: x.reshape(T, Hk, Hv // Hk, dk).sum(2)  # noqa: E731
    return share(gq), share(gk), gv, gg, gb, G, size_g, size_b
