"""The 64-bit definitions of the router and the layer norm: their gradients against
central differences, their choices against brute force."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import router

STEP = 1e-5


def differences(f, x):
    """Central differences of a scalar f at x: an error of order STEP^2 times the
    third derivative, and of 2^-53 |f| / STEP of rounding."""
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        if not np.isfinite(x[i]):
            continue
        a, b = x.copy(), x.copy()
        a[i] += STEP
        b[i] -= STEP
        out[i] = (f(a) - f(b)) / (2 * STEP)
    return out


def logits(rng, rows, experts):
    l = rng.normal(size=(rows, experts))
    l[:, 1] = -np.inf
    l[rows // 2] = -np.inf
    return l


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_gate_gradient_is_the_derivative(score, normalize):
    rng = np.random.default_rng(0)
    l = logits(rng, 6, 7)
    ids = router.choose(l, 3)
    ids[0, 1] = ids[0, 0]  # an expert twice
    ids[1, 2] = -1
    ids[2, 0] = 9
    d = rng.normal(size=ids.shape)
    want = differences(lambda x: (router.gates(x, ids, score, normalize, 2.5) * d).sum(), l)
    np.testing.assert_allclose(router.gate_grad(l, ids, d, score, normalize, 2.5), want, atol=1e-8)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_is_the_derivative(score):
    rng = np.random.default_rng(1)
    l = logits(rng, 6, 7)
    n = router.counts(l, router.choose(l, 2))
    assert n[-1] == 5 and n[:-1].sum() == 10 and n[1] == 0
    want = differences(lambda x: 0.3 * router.balance_loss([x], n, 2, score), l)
    np.testing.assert_allclose(router.balance_grad(l, n, 2, score, 0.3), want, atol=1e-9)


def test_balance_loss_is_one_when_experts_get_alike():
    l = np.log(np.eye(4) * 0.97 + 0.01)
    n = router.counts(l, router.choose(l, 1))
    assert list(n) == [1, 1, 1, 1, 4]
    assert abs(router.balance_loss([l], n, 1, "softmax") - 1.0) < 1e-14


def test_choice_orders_ties_zeros_and_nan():
    l = np.array([[0.0, -0.0, 1.0, 1.0], [np.nan, 2.0, np.inf, -np.inf], [-np.inf] * 4])
    assert router.choose(l, 4).tolist() == [[2, 3, 0, 1], [0, 2, 1, -1], [-1] * 4]


def test_norm_gradients_are_derivatives():
    rng = np.random.default_rng(2)
    x, w, b, d = rng.normal(size=(3, 5)), rng.normal(size=5), rng.normal(size=5), rng.normal(size=(3, 5))
    _, mean, rstd = router.norm(x, w, b, 1e-3)
    dx, dw, db = router.norm_grad(d, x, w, mean, rstd)
    np.testing.assert_allclose(dx, differences(lambda v: (router.norm(v, w, b, 1e-3)[0] * d).sum(), x), atol=1e-8)
    np.testing.assert_allclose(dw, differences(lambda v: (router.norm(x, v, b, 1e-3)[0] * d).sum(), w), atol=1e-8)
    np.testing.assert_allclose(db, differences(lambda v: (router.norm(x, w, v, 1e-3)[0] * d).sum(), b), atol=1e-8)
