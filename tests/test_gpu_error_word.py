"""The device error word: who sets it, what reading it costs, and that no wait of a
long call runs out."""
from __future__ import annotations

import subprocess
import sys

import pytest
import torch

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


def test_each_wait_that_runs_out_sets_its_bit():
    lib = ccl()
    lib.ccl_device_error_flag(clear=True)
    lib.ccl_selftest_bounded_wait()
    torch.cuda.synchronize()
    assert lib.ccl_device_error_flag() == 2 | 4 | 8
    with pytest.raises(lib.CclError) as err:
        lib.ccl_stream_check()
    assert err.value.status == lib.CCL_ERR_TIMEOUT
    assert lib.ccl_device_error_flag() == 0
    a = torch.ones(8, 8, device="cuda", dtype=torch.bfloat16)
    y = torch.empty_like(a)
    lib.ccl_moe_product([a], [torch.tensor([0, 8], device="cuda", dtype=torch.int32)], [a.view(1, 8, 8)], [y])
    lib.ccl_stream_check()
    assert (y == 8).all()


# more stages than two seconds hold, one behind the other in one pair of CTAs:
# by TMA (the loaders' next part is the last row) and by the loaders
@pytest.mark.parametrize("rows,n,k,dtype", [(2 ** 30 + 5, 8, 16, torch.bfloat16), (2 ** 30 + 5, 8, 8, torch.float32),
                                            (2 ** 28 + 5, 7, 9, torch.bfloat16)])
def test_a_sum_of_more_rows_than_a_wait_may_last(rows, n, k, dtype):
    """Mostly zeros: the sums stay whole numbers, whatever their order."""
    lib = ccl()
    lib.ccl_device_error_flag(clear=True)
    x, dy = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda"), torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    at = torch.cat([torch.arange(0, rows, 2 ** 22, device="cuda"), torch.tensor([rows - 1], device="cuda")])
    g = torch.Generator(device="cuda").manual_seed(0)
    a = torch.randint(-1, 2, (len(at), k), generator=g, device="cuda")
    b = torch.randint(-1, 2, (len(at), n), generator=g, device="cuda")
    x[at], dy[at] = a.to(torch.bfloat16), b.to(torch.bfloat16)
    dw = torch.empty(1, n, k, dtype=dtype, device="cuda")
    lib.ccl_moe_product_grad_weight([dy], [x], [torch.tensor([0, rows], dtype=torch.int32, device="cuda")], [dw])
    lib.ccl_stream_check()
    assert torch.equal(dw[0].float(), b.float().T @ a.float())
