"""The layer norm's gradients where the mean is far larger than the deviation.

z = (x - mean) rstd, as the forward pass has it: the difference of two fp32 numbers
and a product, rounded once each, so z is off by 2 roundings of 2^-24 of itself, and
by nothing where x is the mean.  dx and dweight carry that and what test_gpu_norm
counts for their sums (S and T); no term grows with |mean| rstd.
"""
from __future__ import annotations

import numpy as np
import pytest

from gpu_util import ccl
from oracle import router
from test_gpu_norm import STEP, rounded
from test_gpu_router import ONE, Buffer

pytestmark = pytest.mark.gpu

# of each form on the 16-byte grid, then of each off it
WIDTHS = [8, 256, 640, 1024, 4096, 5120, 7168, 8192, 8200, 12288, 61, 401, 1019, 2047, 4095, 8191, 10001]


def rows_of(kind: str, rng, rows: int, cols: int) -> np.ndarray:
    v = rng.normal(size=(rows, cols))
    if kind == "near 4096":
        return v + 4096
    level = rng.uniform(100, 2000, size=rows) * (1.0 if kind == "constant" else 1e31)
    v[1:] = level[1:, None]  # all rows but one
    return v


@pytest.mark.parametrize("dtype,kind,eps", [("f32", "near 4096", 1e-5)] + [(t, *k) for t in ("bf16", "f32") for k in (
    ("constant", 1e-5), ("constant", 1e-12), ("huge", 1e-12))])  # huge: mean * rstd is beyond fp32
@pytest.mark.parametrize("cols", WIDTHS)
def test_gradients_of_rows_far_from_zero(cols, dtype, kind, eps):
    c = ccl()
    rng = np.random.default_rng(cols)
    rows = 5000 if cols <= 256 else 1300 if cols <= 1024 else 330
    x, dy, ds = (rounded(v, dtype) for v in (rows_of(kind, rng, rows, cols), rng.normal(size=(rows, cols)), rng.normal(size=(rows, cols))))
    w = rounded(rng.normal(size=cols), "f32")
    mean, rstd = (s.astype(np.float32) for s in router.norm(x, w, None, eps)[1:])
    assert kind == "near 4096" or (mean[1:] == x[1:, 0]).all()  # z is 0 there
    bx, bd, bs = (Buffer(v.shape, dtype, False, v) for v in (x, dy, ds))
    bw, bm, br = (Buffer(v.shape, "f32", False, v) for v in (w, mean, rstd))
    z = np.abs(x - mean.astype(np.float64)[:, None]) * rstd.astype(np.float64)[:, None]
    g, S, T = np.abs(dy * w), (cols / 32 + 32) * ONE, (rows + 64) * ONE
    for extra in (False, True):
        dx, gw, gb = Buffer(x.shape, dtype), Buffer((cols,), "f32"), Buffer((cols,), "f32")
        c.ccl_layer_norm_grad([bd.t], [bx.t], [bw.t], [bm.t], [br.t], [dx.t], dsum=[bs.t] if extra else None, dweight=[gw.t], dbias=[gb.t])
        want, want_w, want_b = router.norm_grad(dy, x, w, mean, rstd, ds if extra else None)
        bound = rstd[:, None] * (g + g.mean(1, keepdims=True) + z * (g * z).mean(1, keepdims=True)) * (S + 8 * ONE)
        bound = bound + (2 * ONE * np.abs(ds) if extra else 0.0)
        assert (np.abs(dx.numpy() - want) <= bound + STEP[dtype] * np.abs(want)).all()
        assert (np.abs(gw.numpy() - want_w) <= (np.abs(dy) * z).sum(0) * (T + 8 * ONE) + ONE * np.abs(want_w)).all()
        assert (np.abs(gb.numpy() - want_b) <= np.abs(dy).sum(0) * T).all()
