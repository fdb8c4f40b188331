"""fp64 numpy reference of the operators around the step: 8-bit rows, row
norms and their gradients, the linear layer on 8-bit rows.  Written from the
formulas, row by row where that is plainest; shares no code with the library.
"""
from __future__ import annotations

import numpy as np


def rows8(x):
    """(q, scale) of a float matrix.  scale = 2^e, e >= -126 the smallest
    integer with max|row| <= 127 * 2^e; q = x / scale to nearest even."""
    x = np.asarray(x, dtype=np.float64)
    q = np.zeros(x.shape, dtype=np.int8)
    scale = np.empty(x.shape[0], dtype=np.float64)
    for i, row in enumerate(x):
        if not np.all(np.isfinite(row)):
            scale[i] = np.nan
            continue
        top = float(np.max(np.abs(row))) if row.size else 0.0
        e = -126
        if top > 0.0:
            # top / 127 = f 2^k with 0.5 <= f < 1: the power of two at or above it
            f, k = np.frexp(top / 127.0)
            for cand in (int(k) - 1, int(k), int(k) + 1):
                if top <= 127.0 * 2.0 ** cand:
                    e = max(-126, cand)
                    break
        scale[i] = 2.0 ** e
        lim = 63 if e == 122 else 127  # 64 * 2^122 is out of fp32's range
        q[i] = np.clip(np.rint(row / scale[i]), -lim, lim).astype(np.int8)
    return q, scale


def norm_forward(x, gamma, beta, eps, layer=True):
    """(y, mean, rstd)"""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1) if layer else np.zeros(x.shape[0])
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None] * np.asarray(gamma, dtype=np.float64)
    if beta is not None:
        y = y + np.asarray(beta, dtype=np.float64)
    return y, mean, rstd


def norm_backward(dy, x, gamma, mean, rstd, layer=True):
    """(dx, dgamma, dbeta) with the statistics given."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    r = np.asarray(rstd, dtype=np.float64)[:, None]
    m = np.asarray(mean, dtype=np.float64)[:, None] if layer else 0.0
    h = (x - m) * r
    g = dy * np.asarray(gamma, dtype=np.float64)
    dx = g - h * (g * h).mean(axis=1, keepdims=True)
    if layer:
        dx = dx - g.mean(axis=1, keepdims=True)
    return dx * r, (dy * h).sum(axis=0), dy.sum(axis=0)


def restore(q, scale):
    return np.asarray(q, dtype=np.float64) * np.asarray(scale, dtype=np.float64)[:, None]


def linear8_forward(q, scale, wq, wscale, bias=None):
    y = restore(q, scale) @ restore(wq, wscale).T
    return y if bias is None else y + np.asarray(bias, dtype=np.float64)


def linear8_weight_grad(dy, q, scale):
    return np.asarray(dy, dtype=np.float64).T @ restore(q, scale)


def linear8_input_grad(dy, wq, wscale):
    return np.asarray(dy, dtype=np.float64) @ restore(wq, wscale)
