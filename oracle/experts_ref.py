"""fp64 numpy reference of the matrix products grouped by expert, expert by
expert.  Shares no code with the library."""
from __future__ import annotations

import numpy as np


def groups(offsets, rows):
    """(expert, first row, row behind the last) with the offsets held to 0 .. rows."""
    off = [min(max(int(o), 0), rows) for o in offsets]
    return [(e, a, max(a, b)) for e, (a, b) in enumerate(zip(off, off[1:]))]


def forward(x, w, offsets, y):
    """y (rows x out), overwritten where a row belongs to an expert."""
    y = np.array(y, dtype=np.float64)
    for e, a, b in groups(offsets, len(x)):
        y[a:b] = np.asarray(x[a:b], dtype=np.float64) @ np.asarray(w[e], dtype=np.float64).T
    return y


def input_grad(dy, w, offsets, dx):
    dx = np.array(dx, dtype=np.float64)
    for e, a, b in groups(offsets, len(dy)):
        dx[a:b] = np.asarray(dy[a:b], dtype=np.float64) @ np.asarray(w[e], dtype=np.float64)
    return dx


def weight_grad(dy, x, offsets):
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    return np.stack([dy[a:b].T @ x[a:b] for _, a, b in groups(offsets, len(dy))])
