"""float64 definitions of the operators around the layer: layer norm, activations
with a residual, and the gated linear recurrence, with their gradients.

Independent of the CUDA path.  Arrays are numpy float64; features (..., C, T) with
the group index innermost.
"""

from __future__ import annotations

import math

import numpy as np

K0 = math.sqrt(2.0 / math.pi)
K1 = 0.044715


# -------------------------------------------------------------------- layer norm

def norm_forward(x, gamma, beta, eps):
    """y, mean, reciprocal deviation of (N, C, T) features."""
    mu = x.mean(axis=(1, 2))
    d = x - mu[:, None, None]
    r = 1.0 / np.sqrt((d * d).mean(axis=(1, 2)) + eps)
    xh = d * r[:, None, None]
    g = np.ones(x.shape[1]) if gamma is None else gamma
    b = np.zeros(x.shape[1]) if beta is None else beta
    return xh * g[None, :, None] + b[None, :, None], mu, r


def norm_backward(x, dy, gamma, eps):
    """dx, dgamma, dbeta."""
    _, mu, r = norm_forward(x, None, None, eps)
    xh = (x - mu[:, None, None]) * r[:, None, None]
    g = dy if gamma is None else dy * gamma[None, :, None]
    m1 = g.mean(axis=(1, 2), keepdims=True)
    m2 = (g * xh).mean(axis=(1, 2), keepdims=True)
    dx = r[:, None, None] * (g - m1 - xh * m2)
    return dx, (dy * xh).sum(axis=(0, 2)), dy.sum(axis=(0, 2))


# ------------------------------------------------------------------- activations

def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def act(name, z):
    if name == "none":
        return z.copy()
    if name == "relu":
        return np.where(z > 0, z, 0.0)
    if name == "silu":
        return z * _sigmoid(z)
    return 0.5 * z * (1.0 + np.tanh(K0 * (z + K1 * z ** 3)))  # gelu, tanh form


def act_slope(name, z):
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = _sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    t = np.tanh(K0 * (z + K1 * z ** 3))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * K0 * (1.0 + 3.0 * K1 * z * z)


# ---------------------------------------------------------------------- recurrence

def gates(g):
    """a = sigmoid(g) and 1 - a, each without cancellation."""
    return _sigmoid(g), _sigmoid(-g)


def scan_forward(u, g, h0, offsets):
    """u (N, C, T), g (N, C, T) or (N, C), h0 (B, C, T), offsets (B + 1): h, hN.
    Rows of no sequence are zero."""
    if g.ndim < u.ndim:
        g = np.broadcast_to(g[..., None], u.shape)
    a, na = gates(g)
    h, hN = np.zeros_like(u), h0.copy()
    for b in range(len(offsets) - 1):
        for l in range(offsets[b], offsets[b + 1]):
            hN[b] = a[l] * hN[b] + na[l] * u[l]
            h[l] = hN[b]
    return h, hN


def scan_backward(dh, u, g, h0, dhN, offsets):
    """du, dg, dh0."""
    shared = g.ndim < u.ndim
    gf = np.broadcast_to(g[..., None], u.shape) if shared else g
    a, na = gates(gf)
    h, _ = scan_forward(u, g, h0, offsets)
    du, dg, dh0 = np.zeros_like(u), np.zeros_like(u), dhN.copy()
    for b in range(len(offsets) - 1):
        for l in range(offsets[b + 1] - 1, offsets[b] - 1, -1):
            delta = dh[l] + dh0[b]
            before = h[l - 1] if l > offsets[b] else h0[b]
            du[l] = na[l] * delta
            dg[l] = delta * (before - u[l]) * a[l] * na[l]
            dh0[b] = a[l] * delta
    return du, (dg.sum(axis=-1) if shared else dg), dh0
