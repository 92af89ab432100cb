"""AdamW on a tensor of more than 2^32 elements."""
from __future__ import annotations

import pytest
import torch

from gpu_util import ccl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_elements_past_32_bit_indexes(bits):
    """The last 300 elements, from 2^32 on, against a tensor of 300: blocks and
    thresholds repeat after 2^32 elements.  All others have no gradient."""
    ccl()
    from a2a_ring_ordered_gb300.optim import AdamW

    base, tail = 1 << 32, 300
    torch.manual_seed(0)
    p0, g0 = torch.randn(tail, device="cuda").bfloat16(), torch.randn(tail, device="cuda").bfloat16()
    p, g = torch.ones(base + tail, dtype=torch.bfloat16, device="cuda"), torch.zeros(base + tail, dtype=torch.bfloat16, device="cuda")
    p[base:], g[base:] = p0, g0
    small, large = AdamW([p0], [g0], state_bits=bits, weight_decay=0.5, lr=0.25), AdamW([p], [g], state_bits=bits, weight_decay=0.5, lr=0.25)
    for opt in (small, large):
        opt.step()
        opt.step()
    assert torch.equal(p[base:], p0)
    for name, (want,) in small.table.tensors.items():
        if not name.startswith("exp_avg"):
            continue
        got = large.table.tensors[name][0]
        start = base // 128 if name.endswith("scale") else base
        assert torch.equal(got[start:].view(torch.uint8), want.view(torch.uint8))
    for lo in (0, 1 << 31, base - 1000):  # 1 -> 0.875 -> 0.765625: decay alone, in bf16
        assert (p[lo:lo + 1000] == 0.765625).all()
