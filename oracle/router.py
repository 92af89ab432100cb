"""The router's choice, its balance loss and the layer norm from their definitions, in 64 bits.

TEST INFRASTRUCTURE ONLY -- see ``oracle/__init__.py``.

``score`` is "softmax" (u = exp(l)) or "sigmoid" (u = 1 / (1 + exp(-l))); shares are
u over the row's sum.  A masked logit is -inf; a row of them alone chooses nothing
and has no shares.
"""
from __future__ import annotations

import numpy as np


def _scores(logits: np.ndarray, score: str) -> np.ndarray:
    """u over a power of e of its own for each row (a share does not change by it)."""
    l = logits.astype(np.float64)
    top = l.max(axis=1, keepdims=True)
    top[np.isneginf(top)] = 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "softmax":
            return np.exp(l - top)
        low = np.minimum(top, 0.0)
        return np.exp(np.minimum(l, 0.0) - low) / (1.0 + np.exp(-np.abs(l)))


def shares(logits: np.ndarray, score: str) -> np.ndarray:
    u = _scores(logits, score)
    total = u.sum(axis=1, keepdims=True)
    return np.divide(u, total, out=np.zeros_like(u), where=total != 0)


def choose(logits: np.ndarray, k: int) -> np.ndarray:
    """Ids of the k largest logits of each row, largest first, ties by the lower
    index, NaN before all numbers, -1 for -inf."""
    ids = np.full((logits.shape[0], k), -1, dtype=np.int32)
    for t, row in enumerate(logits.astype(np.float64)):
        order = sorted(range(row.size), key=lambda e: (0 if np.isnan(row[e]) else 1, 0.0 if np.isnan(row[e]) else -row[e], e))
        for j, e in enumerate(order[:k]):
            if not np.isneginf(row[e]):
                ids[t, j] = e
    return ids


def _sigmoid(l: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore"):
        return np.where(l >= 0, 1.0 / (1.0 + np.exp(-l)), np.exp(np.minimum(l, 0.0)) / (1.0 + np.exp(np.minimum(l, 0.0))))


def gates(logits: np.ndarray, ids: np.ndarray, score: str, normalize: bool, scale: float) -> np.ndarray:
    there = (ids >= 0) & (ids < logits.shape[1])
    at = np.where(there, ids, 0)
    if normalize:
        u = np.where(there, np.take_along_axis(_scores(logits, score), at, 1), 0.0)
        total = u.sum(axis=1, keepdims=True)
        g = np.divide(u, total, out=np.zeros_like(u), where=total != 0)
    else:
        v = shares(logits, score) if score == "softmax" else _sigmoid(logits.astype(np.float64))
        g = np.take_along_axis(v, at, 1)
    return np.where(there, scale * g, 0.0)


def counts(logits: np.ndarray, ids: np.ndarray) -> np.ndarray:
    """Choices of each expert, then the tokens that have a logit above -inf."""
    experts = logits.shape[1]
    held = ids[(ids >= 0) & (ids < experts)]
    return np.append(np.bincount(held, minlength=experts), (~np.isneginf(logits)).any(axis=1).sum()).astype(np.int64)


def balance_loss(logits: list[np.ndarray], n: np.ndarray, k: int, score: str) -> float:
    """The loss of the tokens of all the given ranks, with their counts n."""
    if n[-1] == 0:
        return 0.0
    total = sum(shares(l, score).sum(axis=0) for l in logits)
    return float((n[:-1] * total).sum() * (len(n) - 1) / (k * float(n[-1]) ** 2))


def gate_grad(logits: np.ndarray, ids: np.ndarray, dgates: np.ndarray, score: str, normalize: bool, scale: float) -> np.ndarray:
    l = logits.astype(np.float64)
    there = (ids >= 0) & (ids < l.shape[1])
    at = np.where(there, ids, 0)
    d = np.where(there, dgates.astype(np.float64), 0.0)
    g = gates(logits, ids, score, normalize, scale)
    out = np.zeros_like(l)
    away = 1.0 if score == "softmax" else _sigmoid(-l)
    if normalize:
        own = g * (d - (g * d).sum(axis=1, keepdims=True) / scale) if scale else 0.0 * g
    else:
        own = g * d
    for t in range(l.shape[0]):
        np.add.at(out[t], at[t][there[t]], own[t][there[t]])
    if score == "softmax" and not normalize:
        out -= shares(logits, score) * own.sum(axis=1, keepdims=True)
    return out * away


def balance_grad(logits: np.ndarray, n: np.ndarray, k: int, score: str, dloss: float) -> np.ndarray:
    p = shares(logits, score)
    # shares add up to 1 (or are all 0), so a constant taken off the counts changes nothing but this function's own rounding
    a = (n[:-1] - n[:-1].mean()) * (dloss * p.shape[1] / (k * float(n[-1]) ** 2)) if n[-1] else 0.0 * n[:-1]
    out = p * (a - (p * a).sum(axis=1, keepdims=True))
    return out if score == "softmax" else out * _sigmoid(-logits.astype(np.float64))


def norm(v: np.ndarray, weight: np.ndarray, bias, eps: float):
    """(y, mean, rstd) of the rows of v."""
    v = v.astype(np.float64)
    mean = v.mean(axis=1)
    rstd = (((v - mean[:, None]) ** 2).mean(axis=1) + eps) ** -0.5
    y = (v - mean[:, None]) * rstd[:, None] * weight.astype(np.float64)
    return (y if bias is None else y + bias.astype(np.float64)), mean, rstd


def norm_grad(dy: np.ndarray, v: np.ndarray, weight: np.ndarray, mean: np.ndarray, rstd: np.ndarray, dsum=None):
    """(dx, dweight, dbias)."""
    d, s = dy.astype(np.float64), rstd.astype(np.float64)[:, None]
    z = (v.astype(np.float64) - mean.astype(np.float64)[:, None]) * s
    g = d * weight.astype(np.float64)
    dx = s * (g - g.mean(axis=1, keepdims=True) - z * (g * z).mean(axis=1, keepdims=True))
    return dx if dsum is None else dx + dsum.astype(np.float64), (d * z).sum(axis=0), d.sum(axis=0)
