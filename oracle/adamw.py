"""One AdamW step, with states in fp32 or in 8 bits (oracle).

TEST INFRASTRUCTURE ONLY -- see ``oracle/__init__.py``.

``step64`` is the formula in 64 bits.  ``step32`` is the same formula with
every operation rounded to fp32 by itself, which is what the library promises
bit for bit; 8-bit states are coded from its results by ``encode_m`` and
``encode_root``, each e4m3 with a scale per 128 elements.
"""
from __future__ import annotations

import numpy as np

from .moe import e4m3_to_f32, f32_to_e4m3

BLOCK = 128
DITHER_ELEM, DITHER_STEP = 1779033703, 2654435769
F = np.float32


def step64(p, g, m, v, step, lr, betas, eps, weight_decay, grad_scale=1.0):
    p, g, m, v = (a.astype(np.float64) for a in (p, g, m, v))
    g = g * grad_scale
    b1, b2 = betas
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    update = (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps) if eps or np.all(v > 0) else None
    return p * (1 - lr * weight_decay) - lr * update, m, v


def step32(p, g, m, v, step, lr, betas, eps, weight_decay, grad_scale=None):
    """(param, m, v, sqrt(v)), all fp32."""
    p, g, m, v = (a.astype(F) for a in (p, g, m, v))
    b1, b2 = betas
    with np.errstate(all="ignore"):
        if grad_scale is not None:
            g = g * F(grad_scale)
        m = m * F(b1) + g * F(1 - b1)
        v = v * F(b2) + (g * g) * F(1 - b2)
        root = np.sqrt(v)
        den = root * F(1.0 / np.sqrt(1 - b2 ** step)) + F(eps)
        p = p * F(1 - lr * weight_decay) - (m / den) * F(lr / (1 - b1 ** step))
    return p, m, v, root


def _blocks(x):
    """x as rows of 128, zeros behind its end."""
    out = np.zeros(-(-x.size // BLOCK) * BLOCK, dtype=F)
    out[:x.size] = x
    return out.reshape(-1, BLOCK)


def _scales(blocks):
    """(factor that codes are made with, scale, whether the block holds anything)."""
    with np.errstate(all="ignore"):
        top = np.where(np.isfinite(blocks), np.abs(blocks), F(0)).max(1, initial=0).astype(F)
        some = top > F(2.0) ** -100
        up = np.where(some, (F(1) / top) * F(448), F(0)).astype(F)
        scale = np.where(some, top * (F(1) / F(448)), F(1)).astype(F)
    return up[:, None], scale, some


def encode_m(m):
    """(codes, scales) of m, to nearest even."""
    b = _blocks(m)
    up, scale, _ = _scales(b)
    with np.errstate(all="ignore"):
        codes = np.where(np.isfinite(b), f32_to_e4m3((b * up).astype(F)), 0x7F).astype(np.uint8)
    return codes.reshape(-1)[:m.size], scale


def thresholds(n: int, step: int) -> np.ndarray:
    """Of each element at this step, in units of 2^-20 of a code's spacing."""
    i = np.arange(n, dtype=np.uint64)
    return ((i * np.uint64(DITHER_ELEM) + np.uint64(step * DITHER_STEP % 2 ** 32)) % np.uint64(2 ** 32)) >> np.uint64(12)


def encode_root(root, v, step):
    """(codes, scales) of sqrt(v): the code below, or the one above where the
    distance to the code below plus the element's threshold reaches a spacing."""
    b = _blocks(root)
    up, scale, some = _scales(b)
    up = np.repeat(up[:, 0], BLOCK)[:root.size]
    some = np.repeat(some, BLOCK)[:root.size]
    codes = np.zeros(root.size, dtype=np.uint8)
    with np.errstate(all="ignore"):
        x = (root * up).astype(F).astype(np.float64)  # in units where 448 is the largest code's value
    fine = np.isfinite(root) & some
    # spacing of the e4m3 numbers at x: 2^-9 up to 2^-6, then 2^(exponent - 3)
    spacing = np.exp2(np.floor(np.log2(np.maximum(np.where(fine, x, 1.0), 2.0 ** -6))) - 3)
    # distances below 2^-20 of the smallest spacing are cut off by the fp32 grid at 2^-149 / 2^-120
    x = np.where(fine, np.rint(x * 2.0 ** 29) / 2.0 ** 29, 0.0)
    at = np.floor(x / spacing + thresholds(root.size, step) / 2.0 ** 20) * spacing
    codes[fine] = f32_to_e4m3(np.minimum(at[fine], 448.0).astype(F))
    codes = np.where(fine & (v > 0), np.maximum(codes, 1), codes)
    return np.where(np.isfinite(root), codes, 0x7F).astype(np.uint8), scale


def decode(codes, scales):
    return (e4m3_to_f32(codes) * np.repeat(scales, BLOCK)[:codes.size]).astype(F)
