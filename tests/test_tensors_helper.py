"""The binding's helper that reads the addresses and sizes of rank buffers."""
from __future__ import annotations

import struct

import pytest
import torch


@pytest.fixture(scope="module")
def helper():
    from a2a_ring_ordered_gb300 import build

    build.build()
    from a2a_ring_ordered_gb300 import ccl as lib

    return lib._TENSORS


def test_what_is_not_a_list_of_gpu_buffers_is_left_to_the_caller(helper):
    t = helper
    host = torch.zeros(2, 3)
    for ts in ([host], (host,), [], [1], [None], "x", None, 7, iter([host]), [host] * 129):
        assert t.ranks(ts, 1, torch.float32, [2], 3) is None
        assert t.shaped(ts, 2, None, None) is None
    assert t.ranks([host], 1, "float32", [2], 3) is None
    assert t.ranks([host], 1, torch.float32, (2,), 3) is None
    assert t.shaped([host], 2, None, "float32") is None
    for bad in (lambda: t.ranks([host]), lambda: t.shaped(), lambda: t.shaped([host], "2", None, None)):
        with pytest.raises(TypeError):
            bad()


@pytest.mark.gpu
def test_addresses_and_sizes_of_gpu_buffers(helper):
    t = helper
    bf = torch.bfloat16
    ts = [torch.zeros(n, 3, 5, dtype=bf, device="cuda") for n in (4, 0, 7)]
    packed = struct.pack("3P", *[x.data_ptr() for x in ts])
    assert t.shaped(ts, 3, 3, bf) == (packed, [4, 0, 7], (3, 5))
    assert t.shaped(tuple(ts), 3, None, None) == (packed, [4, 0, 7], (3, 5))
    assert t.ranks(ts, 3, bf, [4, 0, 7], 15) == packed
    assert t.ranks([torch.nn.Parameter(ts[0])], 1, bf, [4], 15) == packed[:8]
    view = ts[2][2:5]  # contiguous, off its storage's start
    assert t.shaped([view], 3, 1, None) == (struct.pack("P", view.data_ptr()), [3], (3, 5))
    for wrong in ((ts, 2, bf, [4, 0, 7], 15), (ts, 3, torch.float32, [4, 0, 7], 15), (ts, 3, bf, [4, 1, 7], 15), (ts, 3, bf, [4, 0], 15)):
        assert t.ranks(*wrong) is None
    assert t.ranks([ts[0].transpose(1, 2)], 1, bf, [4], 15) is None
    assert t.ranks([ts[0], ts[1].cpu(), ts[2]], 3, bf, [4, 0, 7], 15) is None
    for wrong in ((ts, 2, 3, bf), (ts, 3, 2, bf), (ts, 3, 3, torch.int32), ([ts[0], ts[2][:, :2].contiguous()], 3, None, None),
                  ([ts[0], ts[2].float()], 3, None, None), ([ts[0], ts[2].transpose(1, 2)], 3, None, None), ([ts[0], ts[2].cpu()], 3, None, None),
                  ([torch.zeros((), device="cuda")], 0, None, None)):
        assert t.shaped(*wrong) is None
