"""Plain NumPy definitions of the operators on a token's way through an expert
layer, fp64 where floating point: RMS norm and its gradients, E4M3 tiles, tokens
sorted by expert and returned, microscaled 4-bit values and their products."""
from __future__ import annotations

import numpy as np

from .moe_oracle import e4m3_decode, e4m3_encode


def rmsnorm(x, weight=None, eps=1e-6, residual=None):
    """(o, v, rstd) of v = x + residual, row by row."""
    v = np.asarray(x, np.float64)
    if residual is not None:
        v = v + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt((v ** 2).mean(1) + eps)
    o = v * rstd[:, None]
    return (o if weight is None else o * np.asarray(weight, np.float64)), v, rstd


def rmsnorm_backward(dy, x, rstd, weight=None, dresidual=None):
    """(dx, dweight); x is what was normalized, rstd its."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    rstd = np.asarray(rstd, np.float64)[:, None]
    z = x * rstd
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = rstd * (g - z * (g * z).mean(1, keepdims=True))
    if dresidual is not None:
        dx = dx + np.asarray(dresidual, np.float64)
    return dx, (dy * z).sum(0)


def tiles(o, width=128):
    """(codes, scale) of the rows' tiles of 128 values, the last one shorter."""
    o = np.asarray(o, np.float64)
    n, d = o.shape
    codes, scale = np.zeros((n, d), np.uint8), np.ones((n, -(-d // width)))
    for j, i in enumerate(range(0, d, width)):
        t = o[:, i:i + width]
        amax = np.abs(t).max(1)
        some = amax >= 2.0 ** -100
        scale[some, j] = amax[some] / 448.0
        codes[some, i:i + width] = e4m3_encode(t[some] * (448.0 / amax[some])[:, None])
    return codes, scale


def tile_values(codes, scale, width=128):
    return e4m3_decode(codes) * np.repeat(np.asarray(scale, np.float64), width, 1)[:, :codes.shape[1]]


def dispatch(topk_idx, n_experts, rows=None):
    """(offsets, perm, inv): pair by pair."""
    idx = np.asarray(topk_idx)
    T, K = idx.shape
    rows = T * K if rows is None else rows
    perm, inv = np.full(rows, -1, np.int32), np.full((T, K), -1, np.int32)
    offsets, at = np.zeros(n_experts + 1, np.int32), 0
    for e in range(n_experts):
        for t in range(T):
            for k in range(K):
                if idx[t, k] == e:
                    if at < rows:
                        perm[at], inv[t, k] = t, at
                    at += 1
        offsets[e + 1] = min(at, rows)
    return offsets, perm, inv


def combine(rows, inv, weight=None, base=None):
    rows = np.asarray(rows, np.float64)
    y = np.zeros((inv.shape[0], rows.shape[1])) if base is None else np.array(base, np.float64)
    for t, k in np.ndindex(inv.shape):
        if 0 <= inv[t, k] < len(rows):
            y[t] += rows[inv[t, k]] * (1.0 if weight is None else float(weight[t, k]))
    return y


def combine_backward(dy, rows, inv, weight=None):
    """(drows, dweight); rows that no pair has are NaN."""
    dy, rows = np.asarray(dy, np.float64), np.asarray(rows, np.float64)
    drows, dw = np.full(rows.shape, np.nan), np.zeros(inv.shape)
    for t, k in np.ndindex(inv.shape):
        r = inv[t, k]
        if 0 <= r < len(rows):
            drows[r] = dy[t] * (1.0 if weight is None else float(weight[t, k]))
            dw[t, k] = dy[t] @ rows[r]
    return drows, dw


# ---- microscaled 4-bit values
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32
_HALVES = (E2M1[1:] + E2M1[:-1]) / 2


def mx4_encode(v):
    """(codes [..., k'], bytes [..., k' / 32]) with k' = k filled up with zeros: for
    each value the nearest of the grid, of two equally near ones the even code."""
    v = np.asarray(v, np.float64)
    k = v.shape[-1]
    v = np.concatenate([v, np.zeros((*v.shape[:-1], -k % BLOCK))], -1)
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    amax = np.abs(b).max(-1)
    fine = np.isfinite(amax)
    _, e = np.frexp(np.where(fine & (amax > 0), amax, 1.0))
    e = np.where(amax > 0, np.maximum(e - 3, -127), -127)
    a = np.abs(np.where(fine[..., None], b, 0.0)) * 2.0 ** -e[..., None].astype(np.float64)
    code = np.searchsorted(_HALVES, a, side="left")  # halves go down,
    half = a == _HALVES[np.minimum(code, 6)]
    code = code + (half & (code % 2 == 1))  # unless the code below is odd
    code = np.where(fine[..., None], code + 8 * np.signbit(b), 0)
    return code.reshape(v.shape).astype(np.uint8), np.where(fine, e + 127, 255).astype(np.uint8)


def mx4_decode(codes, byte, k):
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    return (v.reshape(*byte.shape, BLOCK) * s[..., None]).reshape(codes.shape)[..., :k]


def mx4_pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def mx4_unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def mx4_words(byte):
    """Scale bytes [..., rows, blocks] in the kernels' order [..., ceil(blocks / 4), rows, 4]."""
    pad = np.zeros((*byte.shape[:-1], -byte.shape[-1] % 4), np.uint8)
    w = np.concatenate([byte, pad], -1)
    return np.swapaxes(w.reshape(*w.shape[:-1], -1, 4), -3, -2)


def swiglu(x):
    gate, up = np.split(np.asarray(x, np.float64), 2, 1)
    return gate / (1.0 + np.exp(-gate)) * up


def mx4_product(x, w, offsets):
    """(y, sum of |terms|) for values x [rows, k] and w [groups, n, k]; rows outside
    the groups are NaN."""
    y, s = np.full((2, len(x), w.shape[1]), np.nan)
    for g in range(len(w)):
        r = slice(offsets[g], offsets[g + 1])
        y[r], s[r] = x[r] @ w[g].T, np.abs(x[r]) @ np.abs(w[g]).T
    return y, s
