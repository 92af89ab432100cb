"""The experts' products at widths and counts that take other paths of the kernel.

Whole numbers small enough are exact all through and are compared bit by bit.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import ccl
from oracle import experts
from test_gpu_experts import DT, dev, product_inputs, rounded

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    return ccl()


# the last tile of 256 columns is 64, 128, 192 or 256 wide: with 192 each CTA of
# the pair has 96, which do not begin on a multiple of 64
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [[64, 128], [70, 0, 130, 1], [600]])
@pytest.mark.parametrize("n", [128, 192, 256, 320, 448, 704, 960])
@pytest.mark.parametrize("k", [128, 192, 448])
def test_weight_gradient_of_widths_in_64s(lib, n, k, counts, dtype):
    rng = np.random.default_rng(n + k)
    x, w, dy, offsets = product_inputs(rng, counts, n, k, True)
    dw = torch.full(w.shape, 5.0, device="cuda", dtype=DT[dtype])
    lib.ccl_moe_product_grad_weight([dev(dy, BF)], [dev(x, BF)], [dev(offsets)], [dw])
    assert torch.equal(dw.cpu(), rounded(experts.product_grad_weight(dy, x, offsets), DT[dtype]))


@pytest.mark.parametrize("n,k", [(192, 448), (448, 192)])
def test_products_of_widths_in_64s(lib, n, k):
    rng = np.random.default_rng(n)
    x, w, dy, offsets = product_inputs(rng, [70, 0, 192, 1], n, k, True)
    rows = x.shape[0]
    y, dx = torch.zeros(rows, n, dtype=BF, device="cuda"), torch.zeros(rows, k, dtype=BF, device="cuda")
    lib.ccl_moe_product([dev(x, BF)], [dev(offsets)], [dev(w, BF)], [y])
    lib.ccl_moe_product_grad_input([dev(dy, BF)], [dev(offsets)], [dev(w, BF)], [dx])
    assert torch.equal(y.cpu(), rounded(experts.product(x, offsets, w, np.zeros((rows, n))), BF))
    assert torch.equal(dx.cpu(), rounded(experts.product_grad_input(dy, offsets, w, np.zeros((rows, k))), BF))


def test_layer_of_width_192_against_autograd(lib):
    """As the layer's own test (2^-8 per rounded intermediate, in the 2-norm), at
    a width whose weight gradient has 192 columns."""
    from a2a_ring_ordered_gb300.moe_layer import ExpertLayer

    torch.manual_seed(1)
    T, H, F, E, k = 150, 128, 192, 4, 2
    w_up, w_down = (torch.randn(E, F, H, device="cuda") / 11).to(BF), (torch.randn(E, H, F, device="cuda") / 14).to(BF)
    x, dout = [torch.randn(T, H, device="cuda").to(BF)], [torch.randn(T, H, device="cuda").to(BF)]
    ids = [torch.rand(T, E, device="cuda").topk(k, 1).indices.int().contiguous()]
    gates = [torch.rand(T, k, device="cuda")]
    layer = ExpertLayer(w_up, w_down)
    layer.forward(x, ids, gates)
    dw_up, dw_down = [torch.empty(E, F, H, device="cuda")], [torch.empty(E, H, F, device="cuda")]
    layer.backward(dout, dw_up, dw_down)
    X, U, D, G = (t.double().requires_grad_() for t in (x[0], w_up, w_down, gates[0]))
    inner = torch.relu(torch.einsum("tkfh,th->tkf", U[ids[0].long()], X))
    torch.einsum("tk,tkhf,tkf->th", G, D[ids[0].long()], inner).backward(dout[0].double())
    for got, want in ((dw_up[0], U.grad), (dw_down[0], D.grad)):
        assert (got.double() - want).norm() <= 4 * 2.0 ** -8 * want.norm()
