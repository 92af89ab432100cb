"""The AdamW kernel's own square root and quotient on 2^30 pairs of numbers.

With both betas 1/2, no gradient, a learning rate of 1/2 and parameters of zero,
the first step leaves minus the quotient of m / 2 by the denominator, bit for bit.
The reference is torch's on the GPU, whose root and quotient are IEEE's (checked
against numpy's on the first of the numbers)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import ccl
from oracle import adamw

pytestmark = pytest.mark.gpu
H = dict(lr=0.5, betas=(0.5, 0.5), eps=1e-8, weight_decay=0.0)


@pytest.mark.parametrize("low,high", [(0, 2), (-40, 18)])  # exponents of v: every mantissa often; the fast range
def test_quotients(low, high):
    ccl()
    from a2a_ring_ordered_gb300.optim import AdamW

    n = 1 << 24
    g = torch.Generator(device="cuda").manual_seed(high)
    m, v, p = (torch.zeros(n, device="cuda") for _ in range(3))
    opt = AdamW([p], [torch.zeros(n, device="cuda")], **H, states={"exp_avg": [m], "exp_avg_sq": [v]})
    scale = torch.tensor(np.float32(1.0 / np.sqrt(1 - 0.5)), device="cuda")
    eps = torch.tensor(np.float32(1e-8), device="cuda")

    def numbers(lo, hi):
        bits = torch.randint((127 + lo) << 23, (127 + hi) << 23, (n,), generator=g, device="cuda", dtype=torch.int32)
        return bits.view(torch.float32)

    for i in range(32):
        m0, v0 = numbers(-20, 20), numbers(low, high)
        m.copy_(m0)
        v.copy_(v0)
        p.zero_()
        opt.steps = 0
        opt.step()
        want = -((m0 * 0.5) / (torch.sqrt(v0 * 0.5) * scale + eps))
        assert torch.equal(p, want)
        if i == 0:
            k, z = 1 << 18, np.zeros(1 << 18, np.float32)
            of = adamw.step32(z, z, m0[:k].cpu().numpy(), v0[:k].cpu().numpy(), 1, **H)[0]
            np.testing.assert_array_equal(want[:k].cpu().numpy(), of)
