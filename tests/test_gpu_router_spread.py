"""Gates, shares and their gradients of logits that lie far apart, against 64 bits.

The logits are of bf16, or of fp32 on a grid of 2^-8, so that differences of a row
are exact.  In roundings of 2^-24 a score is then off by: the hardware's power of two
(2^-22.5, 3 of them), the factor that its argument's rounding takes (1) and what ln 2
lacks in that (|x| 2^-28, 4 of them at most here); for sigmoid 1 + exp (1), its reciprocal
(2) and their product (1): at most 12.  A share or gate is a score over a sum of scores,
12 each (a sum of scores without that factor, each off by 4/3 |x| and 3 more, is off by
their weighted mean, and that of |x| is at most ln E), with a rounding for each
of the sum's additions (E / 32 a lane and at most 12 to join the lanes), the reciprocal
(2) and the product (1): 40 + E / 32, whatever the distance.  Gradients are sums of
products of two of those with their inputs: twice that of their terms' magnitudes.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import ccl
from oracle import router
from test_gpu_router import ONE, Buffer, grad_terms


def spread_logits(rng, tokens: int, experts: int, dtype: str, top: float) -> np.ndarray:
    """Rows whose largest is about `top`, and which reach 80 below it."""
    l = top - 80.0 * rng.random((tokens, experts)) * rng.random((tokens, 1))
    l = np.round(l * 256) / 256
    l[::5, experts // 2:] = -np.inf
    return torch.tensor(l).to(torch.bfloat16 if dtype == "bf16" else torch.float32).double().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("score,top", [("softmax", 0.0), ("softmax", 40.0), ("sigmoid", 40.0), ("sigmoid", 0.0), ("sigmoid", -60.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts,k", [(4, 2), (8, 2), (16, 4), (32, 8), (60, 6), (128, 8), (256, 8), (256, 12), (384, 8), (1000, 16)])
def test_far_apart(experts, k, dtype, score, top):
    c = ccl()
    rng = np.random.default_rng(experts + k)
    tokens = 2000
    l = spread_logits(rng, tokens, experts, dtype, top)
    tol = (40 + experts / 32) * ONE
    bl, bi, bg = Buffer(l.shape, dtype, False, l), Buffer((tokens, k), "i32"), Buffer((tokens, k), "f32")
    d, dloss = rng.normal(size=(tokens, k)).astype(np.float32), np.float32(0.7)
    want_ids = router.choose(l, k)
    n = router.counts(l, want_ids)
    bd, bn, bdl = Buffer(d.shape, "f32", False, d), Buffer(n.shape, "i32", False, n), Buffer((1,), "f32", False, np.array([dloss]))
    for normalize in (True, False):
        c.ccl_moe_gate([bl.t], [bi.t], [bg.t], score=score, normalize=normalize)
        ids = bi.numpy()
        np.testing.assert_array_equal(ids, want_ids)
        want = router.gates(l, ids, score, normalize, 1.0)
        # what is not normalised underflows to 0 below 2^-126
        assert (np.abs(bg.numpy() - want) <= tol * want + 2.0 ** -126).all()
        for with_loss in (False, True):
            out = Buffer(l.shape, dtype)
            more = dict(counts=[bn.t], dlosses=[bdl.t]) if with_loss else {}
            c.ccl_moe_gate_grad([bl.t], [bi.t], [bd.t], [out.t], score=score, normalize=normalize, **more)
            want, size = grad_terms(l, ids, d, score, normalize, 1.0, n if with_loss else None, k, float(dloss))
            step = 2.0 ** -8 if dtype == "bf16" else ONE
            assert (np.abs(out.numpy() - want) <= 2 * tol * size + step * np.abs(want) + 2.0 ** -124 * (1 + np.abs(d).max())).all()
    out = Buffer(l.shape, dtype)
    c.ccl_moe_balance_grad([bl.t], [bn.t], [out.t], k, score=score, dlosses=[bdl.t])
    want, size = grad_terms(l, ids, None, score, True, 1.0, n, k, float(dloss))
    step = 2.0 ** -8 if dtype == "bf16" else ONE
    assert (np.abs(out.numpy() - want) <= 2 * tol * size + step * np.abs(want) + 2.0 ** -124).all()


@pytest.mark.gpu
@pytest.mark.parametrize("experts", [8, 60, 256, 384])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_stays_a_nan(score, experts):
    """Shares of a row with a NaN are NaN, and so are the loss and gradients made of them;
    the gradient of sigmoid gates is NaN in its column (times 1 - sigmoid), chosen or not."""
    c = ccl()
    torch.manual_seed(0)
    l = torch.randn(30, experts, device="cuda")
    l[3, 1], l[4, 5:] = float("nan"), float("nan")
    ids, d = torch.tensor([[0, 2]] * 30, dtype=torch.int32, device="cuda"), torch.randn(30, 2, device="cuda")
    n, loss, out = torch.empty(experts + 1, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda"), torch.empty_like(l)
    rest = [r for r in range(30) if r not in (3, 4)]
    c.ccl_moe_balance([l], [ids], [n], [loss], score=score)
    assert loss.isnan().all()
    c.ccl_moe_balance_grad([l], [n], [out], 2, score=score)
    assert out[3:5].isnan().all() and out[rest].isfinite().all()
    for normalize in (True, False):
        c.ccl_moe_gate_grad([l], [ids], [d], [out], score=score, normalize=normalize)
        assert out[rest].isfinite().all()
        if score == "sigmoid":
            assert torch.equal(out[3:5].isnan(), l[3:5].isnan())
        else:
            assert out[3:5].isnan().all() if not normalize else out[3:5].isfinite().all()


def test_distances_are_exact():
    """What the tolerances rest on: no difference of a row's logits is rounded in fp32."""
    rng = np.random.default_rng(0)
    for dtype in ("bf16", "f32"):
        for top in (0.0, 40.0, -60.0):
            l = spread_logits(rng, 50, 64, dtype, top).astype(np.float32)
            base = l.max(1, keepdims=True)
            with np.errstate(invalid="ignore"):
                assert ((l - base).astype(np.float64) == l.astype(np.float64) - base.astype(np.float64))[np.isfinite(l)].all()
