"""Plain fp64 NumPy definitions of the operators around the layer: layer norm
and its gradients, products grouped by expert, the orthogonalized update."""
from __future__ import annotations

import numpy as np

NS_COEFFS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7


def layernorm(x, weight=None, bias=None, eps=1e-5, residual=None):
    """(y, v, mean, rstd) of v = x + residual, row by row."""
    v = np.asarray(x, np.float64)
    if residual is not None:
        v = v + np.asarray(residual, np.float64)
    mean = v.mean(1)
    rstd = 1.0 / np.sqrt(((v - mean[:, None]) ** 2).mean(1) + eps)
    y = (v - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, v, mean, rstd


def layernorm_backward(dy, x, mean, rstd, weight=None, dresidual=None):
    """(dx, dweight, dbias); x is what was normalized, mean and rstd its."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    rstd = np.asarray(rstd, np.float64)[:, None]
    z = (x - np.asarray(mean, np.float64)[:, None]) * rstd
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = rstd * (g - g.mean(1, keepdims=True) - z * (g * z).mean(1, keepdims=True))
    if dresidual is not None:
        dx = dx + np.asarray(dresidual, np.float64)
    return dx, (dy * z).sum(0), dy.sum(0)


def grouped(x, w, offsets):
    """y [rows, n] = x W_g^T; rows outside the groups are NaN."""
    y = np.full((len(x), w.shape[1]), np.nan)
    for g in range(len(w)):
        r = slice(offsets[g], offsets[g + 1])
        y[r] = x[r] @ w[g].T
    return y


def grouped_dgrad(dy, w, offsets):
    dx = np.full((len(dy), w.shape[2]), np.nan)
    for g in range(len(w)):
        r = slice(offsets[g], offsets[g + 1])
        dx[r] = dy[r] @ w[g]
    return dx


def grouped_wgrad(dy, x, offsets):
    return np.stack([dy[offsets[g]:offsets[g + 1]].T @ x[offsets[g]:offsets[g + 1]]
                     for g in range(len(offsets) - 1)])


def orthogonalize(grad, momentum_buf=None, momentum=0.95, nesterov=True, steps=5):
    """(out, new momentum) for one matrix."""
    u = np.asarray(grad, np.float64)
    m = None
    if momentum_buf is not None:
        m = momentum * np.asarray(momentum_buf, np.float64) + u
        u = u + momentum * m if nesterov else m
    x = u.T if u.shape[0] > u.shape[1] else u
    x = x / (np.sqrt((x ** 2).sum()) + NS_EPS)
    a, b, c = NS_COEFFS
    for _ in range(steps):
        A = x @ x.T
        x = a * x + (b * A + c * A @ A) @ x
    return (x.T if u.shape[0] > u.shape[1] else x), m
