"""What reading the device error word costs."""
from __future__ import annotations

import subprocess
import sys

import pytest

from conftest import ROOT
from gpu_util import ccl

pytestmark = pytest.mark.gpu

CODE = """
import time, torch
from a2a_ring_ordered_gb300 import ccl
from a2a_ring_ordered_gb300.optim import AdamW

def least():
    best = 1.0
    for _ in range(400):
        t = time.perf_counter()
        ccl.ccl_device_error_flag()
        best = min(best, time.perf_counter() - t)
    return best * 1e6

x = [torch.ones(1000, device="cuda") for _ in range(4)]
ccl.ccl_allreduce(x, [torch.empty_like(t) for t in x])
torch.cuda.synchronize()
before = least()
a = torch.zeros(8, 8, device="cuda", dtype=torch.bfloat16)
ccl.ccl_moe_product([a], [torch.tensor([0, 8], device="cuda", dtype=torch.int32)], [a.view(1, 8, 8)], [torch.empty_like(a)])
AdamW([x[0]], [x[1]], state_bits=8).step()
torch.cuda.synchronize()
print(before, least())
"""


def test_a_process_without_products_and_adamw_reads_one_word():
    """Three words are copied once the kernels that may set the other two have
    been launched, one word before: less than two thirds of the time."""
    ccl()
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    before, after = map(float, r.stdout.split())
    print(f"{before:.1f} us, {after:.1f} us after")
    assert before < after * 2 / 3
