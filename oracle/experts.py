"""A rank's own experts: sort, rows, products and their gradients (oracle).

TEST INFRASTRUCTURE ONLY -- see ``oracle/__init__.py``.

Everything in 64 bits, straight from the definitions: the stable order by
expert, then token, then choice; sorted[row(t, j)] = x[t];
out[t] = sum_j w[t][j] y[row(t, j)] and its gradient; y_e = x_e W_e^T and its
gradients, dx_e = dy_e W_e and dW_e = dy_e^T x_e.
"""
from __future__ import annotations

import numpy as np


def sort(ids: np.ndarray, num_experts: int, first: int = 0):
    """(offsets, rows) of a (tokens, k) array of expert ids."""
    flat = ids.reshape(-1).astype(np.int64) - first
    rows = np.full(flat.size, -1, dtype=np.int32)
    offsets = np.zeros(num_experts + 1, dtype=np.int32)
    at = 0
    for e in range(num_experts):
        mine = np.flatnonzero(flat == e)
        rows[mine] = np.arange(at, at + mine.size)
        at += mine.size
        offsets[e + 1] = at
    return offsets, rows.reshape(ids.shape)


def to_experts(x: np.ndarray, rows: np.ndarray, into: np.ndarray) -> np.ndarray:
    """`into` with the tokens' rows written at their places below its length."""
    out = into.copy()
    for t, j in np.ndindex(rows.shape):
        if 0 <= rows[t, j] < out.shape[0]:
            out[rows[t, j]] = x[t]
    return out


def _terms(y, rows, weights):
    """(value, there, weight) of every choice, 64 bits."""
    there = (rows >= 0) & (rows < y.shape[0])
    picked = np.where(there[..., None], y.astype(np.float64)[np.where(there, rows, 0)] if y.shape[0] else 0.0, 0.0)
    w = np.ones(rows.shape) if weights is None else weights.astype(np.float64)
    return picked, there, np.where(there, w, 0.0)


def from_experts(y, rows, weights):
    """(out, sum of the terms' magnitudes): the second is what rounding errors are measured by."""
    picked, _, w = _terms(y, rows, weights)
    terms = picked * w[..., None]
    return terms.sum(1), np.abs(terms).sum(1)


def from_experts_grad(dout, y, rows, weights, dy_into):
    """(dy, dweights, magnitudes of the dot products' terms)."""
    picked, there, w = _terms(y, rows, weights)
    d = dout.astype(np.float64)
    dy = dy_into.astype(np.float64)
    for t, j in np.argwhere(there):
        dy[rows[t, j]] = w[t, j] * d[t]
    terms = picked * d[:, None, :]
    return dy, terms.sum(-1), np.abs(terms).sum(-1)


def segments(offsets, rows: int):
    """(first, last + 1) row of each expert, cut to the rows there are."""
    out = []
    for e in range(len(offsets) - 1):
        lo = min(max(int(offsets[e]), 0), rows)
        out.append((lo, min(max(int(offsets[e + 1]), lo), rows)))
    return out


def product(x, offsets, w, into):
    y = into.astype(np.float64)
    for e, (lo, hi) in enumerate(segments(offsets, x.shape[0])):
        y[lo:hi] = x[lo:hi].astype(np.float64) @ w[e].astype(np.float64).T
    return y


def product_grad_input(dy, offsets, w, into):
    dx = into.astype(np.float64)
    for e, (lo, hi) in enumerate(segments(offsets, dy.shape[0])):
        dx[lo:hi] = dy[lo:hi].astype(np.float64) @ w[e].astype(np.float64)
    return dx


def product_grad_weight(dy, x, offsets):
    seg = segments(offsets, x.shape[0])
    return np.stack([dy[lo:hi].astype(np.float64).T @ x[lo:hi].astype(np.float64) for lo, hi in seg])
