"""The balance loss of many tokens whose experts are far from alike, against 64 bits.

The column sums of a warp's rows are plain fp32 additions: a rounding each, at most as
many as a warp has rows, and one for each part that is joined, beside the shares' own
(test_gpu_router's).  All terms are positive.
"""
from __future__ import annotations

import pytest
import torch

from gpu_util import ccl
from test_gpu_router import ONE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,experts,k,dt,score", [(16_900_003, 256, 2, torch.bfloat16, "softmax"), (6_000_011, 60, 6, torch.float32, "sigmoid"),
                                                       (9_000_001, 8, 2, torch.bfloat16, "softmax")])
def test_uneven_experts(tokens, experts, k, dt, score):
    c = ccl()
    torch.manual_seed(experts)
    popular = torch.linspace(-3, 3, experts, device="cuda")[torch.randperm(experts, device="cuda")]
    l = torch.empty(tokens, experts, dtype=dt, device="cuda").normal_()
    for at in range(0, tokens, 1 << 20):
        l[at:at + (1 << 20)] += popular.to(dt)
    ids, gates = torch.empty(tokens, k, dtype=torch.int32, device="cuda"), torch.empty(tokens, k, device="cuda")
    counts, loss = torch.empty(experts + 1, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
    c.ccl_moe_gate([l], [ids], [gates], score=score, counts=[counts], losses=[loss])
    again_n, again = torch.empty_like(counts), torch.empty_like(loss)
    c.ccl_moe_balance([l], [ids], [again_n], [again], score=score)
    n, columns = torch.zeros(experts, dtype=torch.int64, device="cuda"), torch.zeros(experts, dtype=torch.float64, device="cuda")
    for at in range(0, tokens, 1 << 20):
        part = l[at:at + (1 << 20)].double()
        u = torch.softmax(part, 1) if score == "softmax" else torch.sigmoid(part)
        columns += (u / u.sum(1, keepdim=True)).sum(0)
        n += torch.bincount(ids[at:at + (1 << 20)].reshape(-1).long(), minlength=experts)
    assert torch.equal(counts[:-1].long(), n) and int(counts[-1]) == tokens and torch.equal(counts, again_n)
    want = float((n.double() * columns).sum() * experts / k / tokens / tokens)
    assert want > 1.5  # far from 1, which alike experts have
    warps = 304 * (16 if experts <= 256 else 8)
    tol = (tokens / warps + 304 + 4 * 16 + experts / 8 + 32) * ONE
    assert abs(float(loss) - want) <= tol * want and abs(float(again) - want) <= tol * want
    print(f"off by {float(loss) / want - 1:.1e} and {float(again) / want - 1:.1e} of {tol:.1e}")
