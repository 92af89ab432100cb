"""The helper that tells whether tensors are where they were."""
from __future__ import annotations

import pytest
import torch


@pytest.fixture(scope="module")
def helper():
    from a2a_ring_ordered_gb300 import build

    build.build()
    from a2a_ring_ordered_gb300 import ccl

    return ccl._TENSORS


def test_tensors_that_stay_and_tensors_that_move(helper):
    a, b, c = torch.zeros(12), torch.zeros(3, 4), torch.zeros(4, 4)
    ts = ((a, b), (c,))
    was = helper.places(ts)
    assert helper.in_place(ts, was) and helper.in_place(ts, helper.places(ts))
    a.add_(1)
    assert helper.in_place(ts, was)
    for change in (lambda: setattr(a, "data", torch.zeros(12)), lambda: setattr(b, "data", b.data.view(torch.int32)),
                   lambda: setattr(b, "data", b.data[:2]), lambda: setattr(c, "data", c.data.T),
                   lambda: a.set_(torch.zeros(13)[1:]), lambda: c.untyped_storage().resize_(0)):
        was = helper.places(ts)
        change()
        assert not helper.in_place(ts, was)


def test_what_is_no_tuple_of_tuples_of_tensors(helper):
    t = torch.zeros(2)
    for wrong in ([t], (t,), ([t],), ((t, 1),), ((None,),), 3, (torch.zeros(2).to_sparse(),), ((torch.zeros(2).to_sparse(),),)):
        with pytest.raises(TypeError):
            helper.places(wrong)
    for wrong in ((), ([t], b""), (((t,),), [1])):
        with pytest.raises(TypeError):
            helper.in_place(*wrong)
    was = helper.places(((t,),))
    assert not helper.in_place(((t, t),), was) and not helper.in_place(((t,),), b"")
    assert helper.places(()) == b"" and helper.in_place((), b"")
