"""The balance loss's part of Router.backward and MoEBlock.backward.

dlogits is rounded to bf16 (2^-8), its own error beside that is what test_gpu_router
allows for a gradient's terms; dx and dweight are sums of its products with bf16
numbers, rounded to bf16 (dx) or held in fp32 with the products' bound (2^-23 times 64
and a little per element).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import ccl
from test_gpu_router import grad_terms, share_tolerance

pytestmark = pytest.mark.gpu


def make(score, together, p=2, T=150, H=64, E=24, k=3):
    ccl()
    from a2a_ring_ordered_gb300.moe_layer import Router

    torch.manual_seed(0)
    router = Router((torch.randn(E, H, device="cuda") / 4).bfloat16(), k, score=score, together=together)
    x = [torch.randn(T - 20 * r, H, device="cuda").bfloat16() for r in range(p)]
    return router, x


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("together", [False, True])
def test_losses_gradients_count_by_themselves(score, together):
    """backward(dlosses=...) takes them at a scale of 1."""
    router, x = make(score, together)
    ids, gates, losses = router.forward(x)
    logits, counts = [v.double().cpu().numpy() for v in router.saved[2]], [v.cpu().numpy() for v in router.saved[4]]
    dlosses = [torch.full((1,), 0.7 - r, device="cuda") for r in range(2)]
    dw = [torch.empty_like(router.weight, dtype=torch.float32) for _ in x]
    dx = router.backward([torch.zeros_like(g) for g in gates], dw, dlosses=dlosses)
    w = router.weight.double().cpu().numpy()
    for r, v in enumerate(x):
        want, size = grad_terms(logits[r], ids[r].cpu().numpy(), None, score, True, 1.0, counts[r], 3, float(dlosses[r]))
        off = 2 * share_tolerance(logits[r]) * size + 2.0 ** -8 * np.abs(want)
        v = v.double().cpu().numpy()
        want_x, want_w = want @ w, want.T @ v
        assert np.abs(want_x).max() > 0 and np.abs(want_w).max() > 0
        terms_x, terms_w = (np.abs(want) + off) @ np.abs(w), (np.abs(want) + off).T @ np.abs(v)
        # bf16 outputs of the products are off by (2048 + ...) 2^-23 of the terms, fp32 ones by 64 and more
        assert (np.abs(dx[r].double().cpu().numpy() - want_x) <= off @ np.abs(w) + 2049 * 2.0 ** -23 * terms_x + 2.0 ** -8 * np.abs(want_x)).all()
        assert (np.abs(dw[r].double().cpu().numpy() - want_w) <= off.T @ np.abs(v) + 65 * 2.0 ** -23 * terms_w).all()


def test_a_scale_is_taken_and_none_is_no_part():
    router, x = make("softmax", False)
    dlosses = [torch.full((1,), 0.5, device="cuda") for _ in x]

    def backward(**kw):
        ids, gates, losses = router.forward(x)
        dw = [torch.empty_like(router.weight, dtype=torch.float32) for _ in x]
        return router.backward([g + 1 for g in gates], dw, **kw) + dw

    def same(a, b):
        return all(torch.equal(u, v) for u, v in zip(a, b))

    nothing = backward()
    assert same(nothing, backward(balance_scale=0.0)) and same(nothing, backward(dlosses=dlosses, balance_scale=0.0))
    assert same(nothing, backward(dlosses=[torch.zeros_like(v) for v in dlosses]))
    whole = backward(dlosses=dlosses)
    assert not same(nothing, whole) and same(whole, backward(dlosses=dlosses, balance_scale=1.0)) and same(whole, backward(balance_scale=0.5))


def test_the_block_hands_the_losses_on():
    c = ccl()
    from a2a_ring_ordered_gb300.moe_layer import ExpertLayer, MoEBlock

    router, x = make("softmax", True)
    E, H = router.weight.shape
    block = MoEBlock(torch.ones(H, device="cuda"), None, router, ExpertLayer((torch.randn(E, 32, H, device="cuda") / 8).bfloat16(),
                                                                            (torch.randn(E, H, 32, device="cuda") / 8).bfloat16()))
    dlosses = [torch.full((1,), 40.0, device="cuda") for _ in x]

    def backward(**kw):
        y, s, losses = block.forward(x)
        new = [[torch.empty(*w.shape, device="cuda") for _ in x] for w in (block.experts.w_up, block.experts.w_down, router.weight, block.norm_weight)]
        return block.backward([torch.ones_like(v) for v in y], None, *new, **kw) + new[2] + new[3]

    whole, again, nothing = backward(dlosses=dlosses), backward(dlosses=dlosses, balance_scale=1.0), backward()
    assert all(torch.equal(a, b) for a, b in zip(whole, again)) and not any(torch.equal(a, b) for a, b in zip(whole, nothing))
    assert c.ccl_device_error_flag() == 0
