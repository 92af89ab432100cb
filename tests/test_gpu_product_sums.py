"""Long sums of the experts' products.

The header's bounds, with S the sum of the terms' magnitudes and L the
contraction's length: an fp32 weight gradient within (64 + L / 512) * 2^-23 * S, a
bf16 output within (2048 + L / 16384) * 2^-23 * S and its rounding, 2^-8 of it.

Terms of one sign are the hard case, for every cut then has the same sign.  A
part of 16384 elements is cut 1024 times by at most 2^-23 of what it has come to,
which is half of it on average: 2^-14 of the result; adding up the parts takes
2^-24 each.  So the MEAN error over many outputs is within 2^-13, where the bf16
roundings of 65,536 outputs average out (2^-8 / sqrt(3) / 256 = 9e-6) once the
outputs are spread by factors.  One sum of 2^20 elements would be off by 1.4e-3.
An fp32 part of 512 rows is cut 32 times by at most 2^-23 of half of it on average:
2^-19, and 2^-19 for the roundings of its 2048 parts, which have both signs: 2^-18.
"""
from __future__ import annotations

import pytest
import torch

from gpu_util import ccl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    return ccl()


def positive(g, rows, cols, spread):
    """Numbers from 1 to 2, times a factor from 1 to 2 of their column (or row)."""
    f = 1 + torch.rand((1, cols) if spread == 1 else (rows, 1), generator=g, device="cuda")
    return ((1 + torch.rand(rows, cols, generator=g, device="cuda")) * f).to(BF)


def check(got, want, size, length):
    """Elementwise by the header's bound, on average by the derived one."""
    err = got.double() - want
    if got.dtype == torch.float32:
        assert (err.abs() <= (64 + length / 512) * 2.0 ** -23 * size).all()
        assert abs((err / want).mean().item()) <= 2.0 ** -18
    else:
        assert (err.abs() <= (2048 + length / 16384) * 2.0 ** -23 * size + 2.0 ** -8 * 1.001 * want.abs()).all()
        assert abs((err / want).mean().item()) <= 2.0 ** -13


# on the 16-byte grid and off it
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rows,n,k", [(2 ** 20, 256, 256), (2 ** 20 - 7, 255, 257)])
def test_weight_gradient_of_many_rows(lib, rows, n, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy = positive(g, rows, k, 1), positive(g, rows, n, 1)
    dw = torch.empty(1, n, k, dtype=dtype, device="cuda")
    lib.ccl_moe_product_grad_weight([dy], [x], [torch.tensor([0, rows], dtype=torch.int32, device="cuda")], [dw])
    want = dy.double().T @ x.double()
    check(dw[0], want, want, rows)


@pytest.mark.parametrize("depth", [2 ** 19, 2 ** 19 - 3])
def test_products_of_long_contractions(lib, depth):
    g = torch.Generator(device="cuda").manual_seed(depth)
    rows = other = 256
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    a, w = positive(g, rows, depth, 0), positive(g, other, depth, 0)
    y = torch.empty(rows, other, dtype=BF, device="cuda")
    lib.ccl_moe_product([a], [off], [w.view(1, other, depth)], [y])
    want = a.double() @ w.double().T
    check(y, want, want, depth)
    wt = w.T.contiguous()
    lib.ccl_moe_product_grad_input([a], [off], [wt.view(1, depth, other)], [y])
    check(y, want, want, depth)


def whole(g, *shape, share):
    """-1, 0 and 1, few enough that sums stay within 256."""
    v = torch.randint(-1, 2, shape, generator=g, device="cuda")
    return torch.where(torch.rand(shape, generator=g, device="cuda") < share, v, 0).to(BF)


# tiles of one part, of two and of three, some of them right after the others;
# lengths at the edges of a part; on the grid and off it
@pytest.mark.parametrize("n,k", [(320, 264), (301, 203)])
def test_parts_of_bf16_weight_gradients(lib, n, k):
    counts = [40000, 3, 16384, 0, 16385, 33000, 500, 32768]
    g = torch.Generator(device="cuda").manual_seed(n)
    x, dy = whole(g, sum(counts), k, share=0.04), whole(g, sum(counts), n, share=0.04)
    off = torch.tensor([0] + counts, dtype=torch.int32, device="cuda").cumsum(0).int()
    dw = torch.full((len(counts), n, k), 7.0, dtype=BF, device="cuda")
    lib.ccl_moe_product_grad_weight([dy], [x], [off], [dw])
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        want = dy[a:b].double().T @ x[a:b].double()
        assert want.numel() == 0 or want.abs().max() <= 256
        assert torch.equal(dw[e].double(), want)


@pytest.mark.parametrize("depth", [16385, 40000, 49153])
def test_parts_of_long_contractions(lib, depth):
    counts, other = [300, 1, 0, 70, 513], 520
    g = torch.Generator(device="cuda").manual_seed(depth)
    rows = sum(counts)
    off = torch.tensor([0] + counts, dtype=torch.int32, device="cuda").cumsum(0).int()
    a, w = whole(g, rows, depth, share=0.04), whole(g, len(counts), other, depth, share=0.04)
    y, dx = torch.full((rows, other), 7.0, dtype=BF, device="cuda"), torch.full((rows, other), 7.0, dtype=BF, device="cuda")
    lib.ccl_moe_product([a], [off], [w], [y])
    lib.ccl_moe_product_grad_input([a], [off], [w.transpose(1, 2).contiguous()], [dx])
    for e, (i, j) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        want = a[i:j].double() @ w[e].double().T
        assert torch.equal(y[i:j].double(), want) and torch.equal(dx[i:j].double(), want)
