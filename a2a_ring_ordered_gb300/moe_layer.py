"""An expert layer on p virtual ranks that hold the same experts, the router that
chooses its experts, and the pre-norm block around both.

Each rank brings its own tokens: rows in expert order (``ccl_moe_sort``,
``ccl_moe_to_experts``), up-projection, ReLU, down-projection
(``ccl_moe_product``), and the gated sum back to the tokens
(``ccl_moe_from_experts``).  The backward pass writes fp32 weight gradients
where the caller wants them, such as the views of ``ddp.GradBuckets``, whose
all-reduce averages them over the ranks.

``Router`` makes the ids and gates from the tokens (a product with one expert's
weights, ``ccl_moe_gate``) with the balance loss, ``MoEBlock`` adds the residual
stream and the layer norm before them (``ccl_layer_norm``).

The products, row moves, norms, choices and sums run in libccl's kernels; torch
allocates the buffers, applies the ReLU and adds the two gradients that reach the
norm.
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


class Router:
    """The k experts of each token, and their gates, by the logits x @ weight.T.

    weight  (experts, hidden) bf16, shared by the ranks.  score, normalize and scale
    as in ``ccl_moe_gate``; ``together``: the balance loss is over all ranks' tokens.

    Logits and their gradients are held in bf16, as ``ccl_moe_product`` makes and takes
    them: of 256 normal ones, four rows in ten have equal ones among the largest nine (one
    in thirteen where eight end), which the lower index wins.  Logits of fp32 go to
    ``ccl_moe_gate`` directly.
    """

    def __init__(self, weight: torch.Tensor, k: int, score: str = "softmax", normalize: bool = True, scale: float = 1.0,
                 together: bool = False):
        if weight.dim() != 2:
            raise ValueError("need weight (experts, hidden)")
        self.weight, self.k = weight, k
        self.how = {"score": score, "normalize": normalize, "scale": scale}
        self.together = together
        self.saved = None

    def forward(self, x: Sequence[torch.Tensor]) -> tuple[list[torch.Tensor], list[torch.Tensor], list[torch.Tensor]]:
        """x[r] (tokens, hidden) bf16 -> (ids, gates, losses): ids[r] (tokens, k) int32,
        gates[r] (tokens, k) fp32 and each rank's balance loss (one fp32)."""
        experts, p, device = self.weight.shape[0], len(x), self.weight.device

        def new(r, n, dtype):
            return torch.empty(x[r].shape[0], n, dtype=dtype, device=device)

        ends = []  # the one expert's rows are all
        for v in x:
            ends.append(torch.zeros(2, dtype=torch.int32, device=device))
            ends[-1][1:].fill_(v.shape[0])
        logits = [new(r, experts, torch.bfloat16) for r in range(p)]
        ccl.ccl_moe_product(list(x), ends, [self.weight[None]] * p, logits)
        ids = [new(r, self.k, torch.int32) for r in range(p)]
        gates = [new(r, self.k, torch.float32) for r in range(p)]
        counts = [torch.empty(experts + 1, dtype=torch.int32, device=device) for _ in x]
        losses = [torch.empty(1, device=device) for _ in x]
        ccl.ccl_moe_gate(logits, ids, gates, **self.how, counts=counts, losses=losses, together=self.together)
        self.saved = (list(x), ends, logits, ids, counts)
        return ids, gates, losses

    def backward(self, dgates: Sequence[torch.Tensor], dweight: Sequence[torch.Tensor], dlosses: Sequence[torch.Tensor] | None = None,
                 balance_scale: float | None = None) -> list[torch.Tensor]:
        """The gradient for x of the last forward: of the gates', and of
        balance_scale * dlosses[r] * losses[r]; writes each rank's weight gradient
        (experts, hidden), fp32 or bf16, into dweight[r].  dlosses None are ones;
        balance_scale None is 1 where dlosses is given, else 0, at which the losses
        have no part."""
        if self.saved is None:
            raise RuntimeError("backward() without a forward()")
        x, ends, logits, ids, counts = self.saved
        self.saved = None
        p = len(x)
        dlogits = [torch.empty_like(v) for v in logits]
        if balance_scale is None:
            balance_scale = 0.0 if dlosses is None else 1.0
        loss = {} if balance_scale == 0 else {"counts": counts, "dlosses": None if dlosses is None else list(dlosses), "balance_scale": balance_scale}
        ccl.ccl_moe_gate_grad(logits, ids, list(dgates), dlogits, **self.how, **loss)
        ccl.ccl_moe_product_grad_weight(dlogits, x, ends, [w[None] for w in dweight])
        dx = [torch.empty_like(v) for v in x]
        ccl.ccl_moe_product_grad_input(dlogits, ends, [self.weight[None]] * p, dx)
        return dx


class MoEBlock:
    """s = x + residual, y = experts(norm(s)): the caller adds y to s, or hands both to
    the next block, whose norm adds them.

    norm_weight, norm_bias  (hidden,) fp32 or bf16, shared by the ranks; the bias may be None.
    """

    def __init__(self, norm_weight: torch.Tensor, norm_bias: torch.Tensor | None, router: Router, experts: ExpertLayer, eps: float = 1e-5):
        self.norm_weight, self.norm_bias, self.router, self.experts, self.eps = norm_weight, norm_bias, router, experts, eps
        self.saved = None

    def forward(self, x: Sequence[torch.Tensor], residual: Sequence[torch.Tensor] | None = None
                ) -> tuple[list[torch.Tensor], list[torch.Tensor], list[torch.Tensor]]:
        """x[r] and residual[r] (tokens, hidden) bf16 -> (y, s, losses); without a
        residual s is x."""
        p = len(x)
        normed = [torch.empty_like(v) for v in x]
        mean, rstd = ([torch.empty(v.shape[0], device=v.device) for v in x] for _ in range(2))
        s = list(x) if residual is None else [torch.empty_like(v) for v in x]
        ccl.ccl_layer_norm(list(x), [self.norm_weight] * p, None if self.norm_bias is None else [self.norm_bias] * p, normed,
                           residual=None if residual is None else list(residual), sum=None if residual is None else s, mean=mean, rstd=rstd,
                           eps=self.eps)
        ids, gates, losses = self.router.forward(normed)
        y = self.experts.forward(normed, ids, gates)
        self.saved = (s, mean, rstd)
        return y, s, losses

    def backward(self, dy: Sequence[torch.Tensor], ds: Sequence[torch.Tensor] | None, dw_up: Sequence[torch.Tensor], dw_down: Sequence[torch.Tensor],
                 dw_router: Sequence[torch.Tensor], dw_norm: Sequence[torch.Tensor], db_norm: Sequence[torch.Tensor] | None = None,
                 dlosses: Sequence[torch.Tensor] | None = None, balance_scale: float | None = None) -> list[torch.Tensor]:
        """The gradient for x (and for residual alike) of the last forward, ds being the
        gradient that reaches s past this block; writes each rank's weight gradients
        where the caller wants them (``ExpertLayer.backward``, ``Router.backward``, the
        norm's (hidden,) fp32 or bf16)."""
        if self.saved is None:
            raise RuntimeError("backward() without a forward()")
        s, mean, rstd = self.saved
        self.saved = None
        dnormed, dgates = self.experts.backward(dy, dw_up, dw_down)
        for d, more in zip(dnormed, self.router.backward(dgates, dw_router, dlosses, balance_scale)):
            d.add_(more)  # both are bf16 already; their sum is rounded to it once more, as the norm takes its gradient
        dx = [torch.empty_like(v) for v in s]
        ccl.ccl_layer_norm_grad(dnormed, s, [self.norm_weight] * len(s), mean, rstd, dx, dsum=None if ds is None else list(ds), dweight=list(dw_norm),
                                dbias=None if db_norm is None else list(db_norm))
        return dx
