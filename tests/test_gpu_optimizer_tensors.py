"""AdamW on tensors whose storage is replaced between steps."""
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


@pytest.mark.parametrize("bits", [32, 8])
def test_a_parameter_with_new_storage_is_the_one_that_is_updated(optim, bits):
    """`p.data = ...` between steps: the step goes on with what p is now."""
    a, pa, _ = one(optim, bits=bits)
    b, pb, gb = one(optim, bits=bits)
    a.step()
    b.step()
    old = pb.data
    kept = old.clone()
    pb.data = old.clone()
    moved = gb.data  # both old storages stay alive to the end of the test
    gb.data = moved.clone()
    moved.zero_()
    a.step()
    b.step()
    assert torch.equal(pa, pb) and torch.equal(old, kept)


def test_a_parameter_without_storage_is_refused(optim):
    opt, p, g = one(optim)
    opt.step()
    bytes_ = p.untyped_storage().nbytes()
    p.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match=r"param\[0\] has lost its storage"):
        opt.step()
    with pytest.raises(ValueError, match="lost its storage"):  # not only the first time
        opt.step()
    assert opt.steps == 1
    p.untyped_storage().resize_(bytes_)
    p.fill_(1)
    opt.step()
    assert opt.steps == 2 and torch.isfinite(p).all()


def test_changed_tensors_are_checked_again(optim):
    opt, p, g = one(optim)
    g.data = g.data.bfloat16()  # a type that serves
    opt.step()
    p.data = torch.ones(999, device="cuda")
    with pytest.raises(ValueError, match="elements"):
        opt.step()
    p.data = torch.ones(1000, 2, device="cuda")[:, 0]
    with pytest.raises(ValueError, match="contiguous"):
        opt.step()
    p.data = torch.ones(1000, device="cuda")
    opt.step()
    assert opt.steps == 2
