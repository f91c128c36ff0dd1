"""fp64 reference of the block norm (gdr_block_norm_fwd, gdr_block_norm_bwd) over rows x [N, d]:

    h = res_scale residual + scale act(gate) w norm(x),   n = w_next next_norm(h)"""
from __future__ import annotations

import numpy as np


def _sigmoid(z):
    return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))


def _act(z, act):
    """The factor and its slope."""
    if z is None:
        return 1.0, 0.0
    if act == "linear":
        return z, np.ones_like(z)
    s = _sigmoid(z)
    return (s, s * _sigmoid(-z)) if act == "sigmoid" else (z * s, s + z * s * _sigmoid(-z))


def _inverse(x, norm, eps):
    """(sum or mean of squares + eps)^(-1/2), 0 where that is 0, and the factor of the sum."""
    if norm in (None, "none"):
        return np.ones(x.shape[:-1] + (1,)), 0.0
    kappa = 1.0 if norm == "l2" else 1.0 / x.shape[-1]
    m = kappa * (x * x).sum(-1, keepdims=True) + eps
    return np.where(m > 0, 1 / np.sqrt(np.where(m > 0, m, 1)), 0.0), kappa


def forward(x, *, norm="rms", weight=None, gate=None, act=None, scale=1.0, residual=None, res_scale=1.0, eps=1e-6,
            next_norm=None, next_weight=None):
    r, _ = _inverse(x, norm, eps)
    h = scale * _act(gate, act)[0] * (r * x * (1.0 if weight is None else weight))
    if residual is not None:
        h = h + res_scale * residual
    if next_norm in (None, "none"):
        return h, None
    return h, _inverse(h, next_norm, eps)[0] * h * (1.0 if next_weight is None else next_weight)


def _through(g, x, r, kappa, w):
    """Gradients of x and of the weight of r w x."""
    t = g if w is None else g * w
    return r * t - kappa * r ** 3 * (t * x).sum(-1, keepdims=True) * x, (g * r * x).sum(0)


def backward(x, dy, *, dn=None, norm="rms", weight=None, gate=None, act=None, scale=1.0, residual=None, res_scale=1.0,
             eps=1e-6, next_norm=None, next_weight=None):
    """(dx, dgate, dresidual, dweight, dnext_weight), None for what is not there."""
    r, kappa = _inverse(x, norm, eps)
    a, slope = _act(gate, act)
    u = r * x * (1.0 if weight is None else weight)
    h = scale * a * u + (0.0 if residual is None else res_scale * residual)
    dh, dw_next = dy, None
    if next_norm not in (None, "none"):
        back, dw_next = _through(dn, h, *_inverse(h, next_norm, eps), next_weight)
        dh = dy + back
    g = scale * dh
    dx, dw = _through(g * a, x, r, kappa, weight)
    return (dx, None if gate is None else g * u * slope, None if residual is None else res_scale * dh,
            None if weight is None else dw, None if next_weight is None else dw_next)
