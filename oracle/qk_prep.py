"""fp64 reference of the query / key preparation and its backward pass (NumPy).
Test infrastructure; shares no code with the HIP library.

A row x of d channels: n = r w x with r = (kappa sum x^2 + eps)^-1/2 (kappa 1 for "l2",
1 / d for "rms"; r = 1 without a norm, 0 where the bracket is 0), then the rotation of the
first 2 len(inv_freq) channels by pos * inv_freq as a d x d matrix, then a scale.
"""
from __future__ import annotations

import numpy as np


def rotation(pos, inv_freq, d, layout, rot_scale=1.0):
    """The rotation of one position as a matrix."""
    R, half = np.eye(d), len(inv_freq)
    for i, f in enumerate(inv_freq):
        e, o = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + half)
        c, s = rot_scale * np.cos(float(pos) * f), rot_scale * np.sin(float(pos) * f)
        R[e, e], R[e, o], R[o, e], R[o, o] = c, -s, s, c
    return R


def _r(x, norm, eps):
    if norm in (None, "none"):
        return np.ones(x.shape[:-1] + (1,))
    m = (x * x).sum(-1, keepdims=True) / (x.shape[-1] if norm == "rms" else 1) + eps
    return np.where(m > 0, 1.0 / np.sqrt(np.where(m > 0, m, 1.0)), 0.0)


def _matrices(B, T, pos, inv_freq, d, layout, rot_scale):
    if inv_freq is None or len(inv_freq) == 0:
        return np.broadcast_to(np.eye(d), (B, T, d, d))
    pos = np.broadcast_to(np.arange(T), (B, T)) if pos is None else pos
    return np.stack([np.stack([rotation(pos[b, t], inv_freq, d, layout, rot_scale) for t in range(T)]) for b in range(B)])


def forward(x, w=None, *, norm="rms", eps=0.0, pos=None, inv_freq=None, layout="half", rot_scale=1.0, scale=1.0):
    """x [B, T, H, d] fp64."""
    B, T, H, d = x.shape
    n = x * _r(x, norm, eps) * (1.0 if w is None else w)
    return scale * np.matmul(n, _matrices(B, T, pos, inv_freq, d, layout, rot_scale).transpose(0, 1, 3, 2))


def backward(x, g, w=None, *, norm="rms", eps=0.0, pos=None, inv_freq=None, layout="half", rot_scale=1.0, scale=1.0):
    """Gradients (dx, dw) of sum(forward(x, w) g)."""
    B, T, H, d = x.shape
    m = scale * np.matmul(g, _matrices(B, T, pos, inv_freq, d, layout, rot_scale))
    r = _r(x, norm, eps)
    t = m * (1.0 if w is None else w)
    kappa = {"rms": 1.0 / d, "l2": 1.0}.get(norm, 0.0)
    dx = r * t - kappa * r ** 3 * (t * x).sum(-1, keepdims=True) * x
    return dx, (m * r * x).sum((0, 1, 2))
