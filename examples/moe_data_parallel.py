"""Trains one mixture-of-experts layer on p data-parallel virtual ranks.

Every rank routes its own tokens to the same experts; the router's and the experts'
weight gradients are written straight into the DDP buckets, each bucket's ring-ordered
all-reduce averages them over the ranks and rounds them to bf16, and AdamW, with
its moments in 8 bits, updates fp32 master weights and the bf16 copies that the
next forward pass reads.

    python examples/moe_data_parallel.py [--ranks 4] [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def train(ranks: int = 4, steps: int = 60, tokens: int = 512, hidden: int = 256, width: int = 512, experts: int = 16, k: int = 2,
          state_bits: int = 8, seed: int = 0) -> list[float]:
    """Losses of each step: the layer learns another layer of its shape."""
    from a2a_ring_ordered_gb300.ddp import GradBuckets
    from a2a_ring_ordered_gb300.moe_layer import ExpertLayer, Router
    from a2a_ring_ordered_gb300.optim import AdamW

    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev) * scale

    shapes = [(experts, hidden), (experts, width, hidden), (experts, hidden, width)]  # router, up, down
    masters = [normal(*s, scale=s[-1] ** -0.5) for s in shapes]
    weights = [m.bfloat16() for m in masters]
    buckets = GradBuckets(shapes, ranks, dev)
    optimizer = AdamW(masters, [buckets.averaged(0, i) for i in range(3)], lr=2e-3, betas=(0.9, 0.98), weight_decay=0.0,
                      state_bits=state_bits, copies=weights)
    router, layer = Router(weights[0], k), ExpertLayer(weights[1], weights[2])
    target = ExpertLayer(normal(*shapes[1], scale=hidden ** -0.5).bfloat16(), normal(*shapes[2], scale=width ** -0.5).bfloat16())

    x = [normal(tokens, hidden).bfloat16() for _ in range(ranks)]
    want = target.forward(x, *Router(normal(experts, hidden).bfloat16(), k).forward(x)[:2])
    losses = []
    for _ in range(steps):
        ids, gates, _ = router.forward(x)
        out = layer.forward(x, ids, gates)
        errors = [o.float() - t.float() for o, t in zip(out, want)]
        losses.append(sum(e.square().mean() for e in errors) / ranks)
        dout = [(e * (2.0 / e.numel())).bfloat16() for e in errors]
        _, dgates = layer.backward(dout, [buckets.grad(r, 1) for r in range(ranks)], [buckets.grad(r, 2) for r in range(ranks)])
        router.backward(dgates, [buckets.grad(r, 0) for r in range(ranks)])
        for b in range(buckets.num_buckets):
            buckets.reduce_bucket(b)
        optimizer.step()
    return [float(v) for v in losses]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    for i, loss in enumerate(train(a.ranks, a.steps, state_bits=a.state_bits)):
        if i % 10 == 0 or i == a.steps - 1:
            print(f"step {i:4d}  loss {loss:.5f}")


if __name__ == "__main__":
    main()
