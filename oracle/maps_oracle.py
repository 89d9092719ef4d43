"""fp64 CPU oracle of the plain linear maps (4-bit weights, experts' maps) and
of the grouping around them (test infrastructure, like gsi_oracle: the library
never calls it and shares no code with it).

Every function is a loop or a numpy product over the definition in gsi.h.
"""
from __future__ import annotations

import numpy as np


def q4_weights(codes, scales, zeros, group: int) -> np.ndarray:
    """W [d_out][d] = scale (code - zero) from codes [d_out][d / 2] (even
    column in the low nibble); zeros None is 8."""
    codes = np.asarray(codes).astype(np.int64)
    d_out, half = codes.shape
    W = np.empty((d_out, 2 * half))
    for c in range(2 * half):
        nibble = codes[:, c // 2] // 16 if c % 2 else codes[:, c // 2] % 16
        z = 8 if zeros is None else np.asarray(zeros).astype(np.int64)[:, c // group] % 16
        W[:, c] = np.asarray(scales, dtype=np.float64)[:, c // group] * (nibble - z)
    return W


def grouped_linear(W, x, offsets, rows, y) -> np.ndarray:
    """y with the rows of every expert replaced: y[r] = W[e] x[rows[r]], zeros
    where rows[r] names no row of x; W a list of [d_out][d]."""
    y = np.array(y, dtype=np.float64)
    x = np.asarray(x, dtype=np.float64)
    for e in range(len(W)):
        for r in range(int(offsets[e]), int(offsets[e + 1])):
            src = r if rows is None else int(rows[r])
            y[r] = np.asarray(W[e], dtype=np.float64) @ x[src] if 0 <= src < len(x) else 0.0
    return y


def group_rows(ids, n: int):
    """(offsets, rows, pos) of gsi_group_rows."""
    ids = np.asarray(ids)
    T, top = ids.shape
    offsets, rows = [0], []
    pos = np.full((T, top), -1, dtype=np.int32)
    for e in range(n):
        for t, j in zip(*np.nonzero(ids == e)):
            pos[t, j] = len(rows)
            rows.append(t)
        offsets.append(len(rows))
    rows += [-1] * (T * top - len(rows))
    return np.array(offsets, np.int32), np.array(rows, np.int32), pos


def group_combine(y, pos, weights, base) -> np.ndarray:
    """out[t] = base[t] + sum_j weights[t][j] y[pos[t][j]]."""
    y = np.asarray(y, dtype=np.float64)
    T, top = np.asarray(pos).shape
    out = np.zeros((T, y.shape[1])) if base is None else np.array(base, dtype=np.float64)
    for t in range(T):
        for j in range(top):
            p = int(pos[t][j])
            if 0 <= p < len(y):
                out[t] += (1.0 if weights is None else float(weights[t][j])) * y[p]
    return out
