"""The library is built without torch, and the binding works without its compiled helper."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from conftest import ROOT

WITHOUT = """
import os, warnings
exists = os.path.exists
os.path.exists = lambda p: exists(p) and not str(p).endswith("_tensors.so")
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    from a2a_ring_ordered_gb300 import ccl
os.path.exists = exists
assert any("_tensors.so" in str(w.message) for w in said), [str(w.message) for w in said]
"""


def without_helper(code: str) -> None:
    r = subprocess.run([sys.executable, "-c", WITHOUT + code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.fixture(scope="module")
def built():
    from a2a_ring_ordered_gb300 import build

    build.build()
    return build


def test_library_is_built_without_torch(built, monkeypatch):
    def none():
        raise RuntimeError("torch is required to build _tensors.so")

    monkeypatch.setattr(built, "_torch", none)
    with pytest.warns(RuntimeWarning, match="torch is required"):
        assert built.build() == built.LIB


def test_import_and_refusals_without_the_helper(built):
    without_helper("""
import torch
print(ccl.ccl_chunk_bounds(4, 10, 1))
for call in (lambda: ccl.ccl_moe_sort([torch.zeros(2, 2)], 4, [], []), lambda: ccl.ccl_moe_product([3], [], [], [])):
    try:
        call()
    except ValueError as e:
        assert "must be a CUDA tensor" in str(e), e
    else:
        raise SystemExit("not refused")
""")


def test_a_file_that_is_no_helper_is_not_used(built, tmp_path):
    from a2a_ring_ordered_gb300 import ccl

    bad = tmp_path / "_tensors.so"
    bad.write_bytes(b"not a library")
    with pytest.warns(RuntimeWarning, match="is not used"):
        assert ccl._load_tensors(str(bad)) is ccl._PlainTensors


def test_places_without_the_helper(built):
    from a2a_ring_ordered_gb300.ccl import _PlainTensors as plain

    a, b = torch.zeros(12), torch.zeros(4, 4)
    ts = ((a,), (b,))
    was = plain.places(ts)
    a.add_(1)
    assert plain.in_place(ts, was) and not plain.in_place(ts, b"")
    for change in (lambda: setattr(a, "data", torch.zeros(12)), lambda: setattr(b, "data", b.data.T), lambda: b.untyped_storage().resize_(0)):
        was = plain.places(ts)
        change()
        assert not plain.in_place(ts, was)


@pytest.mark.gpu
def test_calls_without_the_helper(built):
    without_helper(f"""
import sys, torch
sys.path.insert(0, {os.path.join(ROOT, "tests")!r})
from a2a_ring_ordered_gb300.moe_layer import ExpertLayer
from a2a_ring_ordered_gb300.optim import AdamW
assert ccl._TENSORS is ccl._PlainTensors
torch.manual_seed(0)
w = [torch.randn(4, 24, 16, device="cuda").bfloat16(), torch.randn(4, 16, 24, device="cuda").bfloat16()]
x, ids = [torch.randn(30, 16, device="cuda").bfloat16()] * 2, [torch.randint(4, (30, 2), device="cuda", dtype=torch.int32)] * 2
gates = [torch.rand(30, 2, device="cuda")] * 2
layer = ExpertLayer(*w)
out = layer.forward(x, ids, gates)
grads = [[torch.empty(v.shape, device="cuda") for _ in x] for v in w]
dx, dgates = layer.backward(out, *grads)
U, D, X = (v.float() for v in (*w, x[0]))
up = torch.relu(torch.einsum("tkfh,th->tkf", U[ids[0].long()], X))
want = torch.einsum("tk,tkhf,tkf->th", gates[0], D[ids[0].long()], up)
for o in out:
    assert (o.float() - want).norm() < 0.02 * want.norm()
p = torch.ones(10, device="cuda")
opt = AdamW([p], [torch.ones(10, device="cuda")])
opt.step()
p.data = torch.ones(10, device="cuda")
opt.step()
assert (p < 1).all()
""")
