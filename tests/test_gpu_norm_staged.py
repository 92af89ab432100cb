"""The layer norm where weights go through shared memory: calls of four rows and more for
each group of each CTA, which are 1824 of 512 / 256 / ... threads in groups of 32 to 512.
Tolerances as in test_gpu_norm."""
from __future__ import annotations

import pytest
import torch

from gpu_util import ccl
from test_gpu_router_scale import check_norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("dt,wt", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("rows,cols", [(58_500, 256), (58_500, 1024), (30_000, 2048), (7400, 7168), (7400, 8200), (7400, 12_288), (7400, 16_384)])
def test_rows_enough_to_stage(rows, cols, dt, wt, residual):
    """8 groups a CTA to 1024 columns of bf16, 4 at 2048, fewer of fp32, 1 from 4096 on;
    16,384 columns with a bias take all of 128 KB."""
    c = ccl()
    torch.manual_seed(cols)
    x, more = (torch.randn(rows, cols, device="cuda", dtype=dt) + a for a in (0.5, 0.25))
    for off in (0, 1):  # weights on the 16-byte grid and off it
        w, b = (torch.randn(cols + off, device="cuda").to(wt)[off:] for _ in range(2))
        for bias in (b, None):
            y, total = torch.empty_like(x), torch.full_like(x, 7.0) if residual else None
            c.ccl_layer_norm([x], [w], None if bias is None else [bias], [y], residual=[more] if residual else None, sum=[total] if residual else None)
            if residual:
                assert torch.equal(total, (x.float() + more.float()).to(dt))
            for part in (slice(0, rows // 2), slice(rows // 2, rows)):
                check_norm(y[part], (total if residual else x)[part], w, bias, 1e-5)


def test_ranks_of_their_own_weights():
    """A CTA stages its own rank's weights; ranks of many rows, of one and of none."""
    c = ccl()
    torch.manual_seed(0)
    rows, cols = [9000, 1, 0, 6000], 7168
    x, more = ([torch.randn(t, cols, device="cuda").bfloat16() for t in rows] for _ in range(2))
    w, b = ([torch.randn(cols, device="cuda") for _ in rows] for _ in range(2))
    y, total = ([torch.empty_like(v) for v in x] for _ in range(2))
    mean, rstd = ([torch.empty(t, device="cuda") for t in rows] for _ in range(2))
    c.ccl_layer_norm(x, w, b, y, residual=more, sum=total, mean=mean, rstd=rstd)
    for r, t in enumerate(rows):
        assert torch.equal(total[r], (x[r].float() + more[r].float()).bfloat16())
        if t:
            check_norm(y[r], total[r], w[r], b[r], 1e-5)
