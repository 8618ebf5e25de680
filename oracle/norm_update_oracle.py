"""Float64 definitions of the layer norm, its gradient, the Newton-Schulz
orthogonalisation and the Muon update (numpy, test infrastructure)."""
from __future__ import annotations

import numpy as np

COEFS = (3.4445, -4.7750, 2.0315)


def layer_norm(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd) of the rows of x."""
    x = np.asarray(x, np.float64)
    mean = x.sum(-1, keepdims=True) / x.shape[-1]
    var = ((x - mean) ** 2).sum(-1, keepdims=True) / x.shape[-1]
    rstd = 1.0 / np.sqrt(var + eps)
    y = (x - mean) * rstd
    if gamma is not None:
        y = y * np.asarray(gamma, np.float64)
    if beta is not None:
        y = y + np.asarray(beta, np.float64)
    return y, mean[..., 0], rstd[..., 0]


def layer_norm_backward(x, dy, gamma, mean, rstd, dres=None):
    """(dx, dgamma, dbeta) for given row statistics."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    h = (x - np.asarray(mean, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    D = x.shape[1]
    dx = np.asarray(rstd, np.float64)[:, None] * (
        g - g.sum(1, keepdims=True) / D - h * (g * h).sum(1, keepdims=True) / D)
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    return dx, (dy * h).sum(0), dy.sum(0)


def orthogonalize(g, steps=5, eps=1e-7):
    """Newton-Schulz orthogonalisation of one matrix, step by step."""
    x = np.asarray(g, np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    a, b, c = COEFS
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.T if tall else x


def muon_update(g, momentum, w, lr, mu=0.95, weight_decay=0.0, scale=1.0, nesterov=True, steps=5,
                eps=1e-7):
    """(momentum, w) after one step on one matrix."""
    g, w = np.asarray(g, np.float64), np.asarray(w, np.float64)
    m = mu * np.asarray(momentum, np.float64) + g
    u = g + mu * m if nesterov else m
    return m, (1.0 - lr * weight_decay) * w - lr * scale * orthogonalize(u, steps, eps)
