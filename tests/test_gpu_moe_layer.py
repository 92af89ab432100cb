"""The expert layer, and the training example that runs the new operators together."""
from __future__ import annotations

import os
import sys

import pytest
import torch

from conftest import ROOT
from gpu_util import ccl

pytestmark = pytest.mark.gpu


def test_layer_and_its_gradients_against_autograd():
    """Against the same layer in 64 bits on the same bf16 inputs.  Each stored
    intermediate is rounded to bf16 once (2^-8): up, y, dy, dup and dxs; in the
    2-norm, with errors that add up rather than cancel, forward takes three of
    them (up, y, out), dx five more, weight gradients three; ReLU's derivative
    follows the rounded up-projection, whose sign a rounding does not change."""
    ccl()
    from a2a_ring_ordered_gb300.moe_layer import ExpertLayer

    torch.manual_seed(0)
    p, T, H, F, E, k = 2, 200, 96, 160, 6, 3
    w_up, w_down = (torch.randn(E, F, H, device="cuda") / 10).bfloat16(), (torch.randn(E, H, F, device="cuda") / 12).bfloat16()
    x = [torch.randn(T, H, device="cuda").bfloat16() for _ in range(p)]
    ids = [torch.rand(T, E, device="cuda").topk(k, 1).indices.int().contiguous() for _ in range(p)]
    gates = [torch.rand(T, k, device="cuda") for _ in range(p)]
    layer = ExpertLayer(w_up, w_down)
    out = layer.forward(x, ids, gates)
    dout = [torch.randn(T, H, device="cuda").bfloat16() for _ in range(p)]
    dw_up, dw_down = [torch.empty(E, F, H, device="cuda") for _ in range(p)], [torch.empty(E, H, F, device="cuda") for _ in range(p)]
    dx, dgates = layer.backward(dout, dw_up, dw_down)

    def near(got, want, roundings):
        assert (got.double() - want).norm() <= roundings * 2.0 ** -8 * want.norm()

    for r in range(p):
        X, U, D, G = (t.double().requires_grad_() for t in (x[r], w_up, w_down, gates[r]))
        hidden = torch.relu(torch.einsum("tkfh,th->tkf", U[ids[r].long()], X))
        want = torch.einsum("tk,tkhf,tkf->th", G, D[ids[r].long()], hidden)
        want.backward(dout[r].double())
        near(out[r], want.detach(), 3)
        near(dx[r], X.grad, 8)
        near(dgates[r], G.grad, 3)
        near(dw_up[r], U.grad, 4)
        near(dw_down[r], D.grad, 4)
    with pytest.raises(RuntimeError, match="without a forward"):
        layer.backward(dout, dw_up, dw_down)


@pytest.mark.parametrize("state_bits", [8, 32])
def test_example_learns(state_bits):
    ccl()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_data_parallel

    losses = moe_data_parallel.train(ranks=3, steps=40, tokens=256, hidden=128, width=192, experts=8, state_bits=state_bits)
    assert all(v == v for v in losses) and losses[-1] < 0.7 * losses[0]
