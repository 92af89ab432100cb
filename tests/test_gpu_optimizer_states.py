"""States that an AdamW takes over: other shapes, other types."""
from __future__ import annotations

import pytest
import torch

from gpu_util import ccl

pytestmark = pytest.mark.gpu
H = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def optim():
    ccl()
    from a2a_ring_ordered_gb300 import optim as mod

    return mod


def one(optim, n=1000, bits=32):
    torch.manual_seed(0)
    p, g = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
    return optim.AdamW([p], [g], **H, state_bits=bits), p, g


def test_states_of_another_shape_are_taken_over(optim):
    a, pa, _ = one(optim)
    a.step()
    m = [torch.zeros(10, 100, device="cuda") for _ in range(2)]
    p, g = torch.zeros(10, 100, device="cuda"), torch.ones(10, 100, device="cuda")
    b = optim.AdamW([p], [g], **H, states={"exp_avg": [m[0]], "exp_avg_sq": [m[1]]})
    b.load_state_dict(a.state_dict())
    assert torch.equal(m[0].view(-1), a.moments(0)[0]) and b.steps == 1


def test_states_of_another_type_are_refused_before_any_is_taken(optim):
    a, _, _ = one(optim)
    a.step()
    b, _, _ = one(optim)
    for wrong in (torch.float64, torch.int32, torch.bfloat16):
        state = a.state_dict()
        state["states"]["exp_avg_sq"][0] = state["states"]["exp_avg_sq"][0].to(wrong)
        with pytest.raises(ValueError, match="exp_avg_sq"):
            b.load_state_dict(state)
        assert b.steps == 0 and (b.moments(0)[0] == 0).all() and (b.moments(0)[1] == 0).all()


@pytest.mark.parametrize("kind", [torch.uint8, torch.float8_e4m3fn])
def test_codes_are_taken_over_from_either_type(optim, kind):
    a, _, _ = one(optim, bits=8)
    a.step()
    b, _, _ = one(optim, bits=8)
    state = a.state_dict()
    for name in ("exp_avg", "exp_avg_sq"):
        state["states"][name] = [t.view(kind) for t in state["states"][name]]
    b.load_state_dict(state)
    for name, ts in a.table.tensors.items():
        if name.startswith("exp_avg"):
            assert torch.equal(ts[0].view(torch.uint8), b.table.tensors[name][0].view(torch.uint8))
