"""An expert layer on p virtual ranks that hold the same experts.

Each rank brings its own tokens: rows in expert order (``ccl_moe_sort``,
``ccl_moe_to_experts``), up-projection, ReLU, down-projection
(``ccl_moe_product``), and the gated sum back to the tokens
(``ccl_moe_from_experts``).  The backward pass writes fp32 weight gradients
where the caller wants them, such as the views of ``ddp.GradBuckets``, whose
all-reduce averages them over the ranks.

The products, row moves and sums run in libccl's kernels; torch allocates the
buffers and applies the ReLU.
"""
from __future__ import annotations

from typing import Sequence

import torch

from . import ccl


class ExpertLayer:
    """out[t] = sum_j gates[t, j] * w_down[e] @ relu(w_up[e] @ x[t]), e = ids[t, j].

    w_up    (experts, width, hidden) bf16, shared by the ranks.
    w_down  (experts, hidden, width) bf16.
    """

    def __init__(self, w_up: torch.Tensor, w_down: torch.Tensor):
        if w_up.dim() != 3 or w_down.shape != (w_up.shape[0], w_up.shape[2], w_up.shape[1]):
            raise ValueError("need w_up (experts, width, hidden) and w_down (experts, hidden, width)")
        self.w_up, self.w_down = w_up, w_down
        self.saved = None

    def forward(self, x: Sequence[torch.Tensor], ids: Sequence[torch.Tensor],
                gates: Sequence[torch.Tensor]) -> list[torch.Tensor]:
        """x[r] (tokens, hidden) bf16, ids[r] (tokens, k) int32, gates[r] (tokens, k) fp32."""
        experts, width, hidden = self.w_up.shape
        p, device = len(x), self.w_up.device

        def rows(r, n):
            return torch.empty(ids[r].numel(), n, dtype=torch.bfloat16, device=device)

        offsets = [torch.empty(experts + 1, dtype=torch.int32, device=device) for _ in range(p)]
        places = [torch.empty_like(i) for i in ids]
        xs, up, y = ([rows(r, n) for r in range(p)] for n in (hidden, width, hidden))
        out = [torch.empty_like(v) for v in x]
        ccl.ccl_moe_sort(list(ids), experts, offsets, places)
        ccl.ccl_moe_to_experts(list(x), places, xs)
        ccl.ccl_moe_product(xs, offsets, [self.w_up] * p, up)
        for v in up:
            v.relu_()
        ccl.ccl_moe_product(up, offsets, [self.w_down] * p, y)
        ccl.ccl_moe_from_experts(y, places, list(gates), out)
        self.saved = (offsets, places, list(gates), xs, up, y)
        return out

    def backward(self, dout: Sequence[torch.Tensor], dw_up: Sequence[torch.Tensor],
                 dw_down: Sequence[torch.Tensor]) -> tuple[list[torch.Tensor], list[torch.Tensor]]:
        """Gradients of the last forward: returns (dx, dgates) and writes each
        rank's weight gradients (fp32 or bf16) into dw_up[r] and dw_down[r]."""
        if self.saved is None:
            raise RuntimeError("backward() without a forward()")
        offsets, places, gates, xs, up, y = self.saved
        self.saved = None
        p = len(xs)
        dy = [torch.empty_like(v) for v in y]
        dgates = [torch.empty_like(g) for g in gates]
        ccl.ccl_moe_from_experts_grad(list(dout), y, places, gates, dy, dgates)
        dup = [torch.empty_like(v) for v in up]
        ccl.ccl_moe_product_grad_input(dy, offsets, [self.w_down] * p, dup)
        ccl.ccl_moe_product_grad_weight(dy, up, offsets, list(dw_down))
        for d, v in zip(dup, up):
            d.masked_fill_(v <= 0, 0)
        ccl.ccl_moe_product_grad_weight(dup, xs, offsets, list(dw_up))
        dxs = [torch.empty_like(v) for v in xs]
        ccl.ccl_moe_product_grad_input(dup, offsets, [self.w_up] * p, dxs)
        dx = [torch.empty_like(d) for d in dout]
        ccl.ccl_moe_from_experts(dxs, places, None, dx)
        return dx, dgates
