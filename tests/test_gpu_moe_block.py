"""The norm, the router and the expert layer together, against autograd in 64 bits."""
from __future__ import annotations

import pytest
import torch

from gpu_util import ccl

pytestmark = pytest.mark.gpu


def make(p, T, H, F, E, k, score, together):
    from a2a_ring_ordered_gb300.moe_layer import ExpertLayer, MoEBlock, Router

    w_up, w_down = (torch.randn(E, F, H, device="cuda") / H ** 0.5).bfloat16(), (torch.randn(E, H, F, device="cuda") / F ** 0.5).bfloat16()
    w_router = (torch.randn(E, H, device="cuda") / H ** 0.5).bfloat16()
    w_norm, b_norm = torch.randn(H, device="cuda") * 0.2 + 1, torch.randn(H, device="cuda") * 0.1
    router = Router(w_router, k, score=score, scale=1.5, together=together)
    return MoEBlock(w_norm, b_norm, router, ExpertLayer(w_up, w_down)), (w_up, w_down, w_router, w_norm, b_norm)


@pytest.mark.parametrize("score,together,residual", [("softmax", False, True), ("sigmoid", True, True), ("softmax", True, False)])
def test_block_and_its_gradients(score, together, residual):
    """bf16 intermediates are rounded once each, 2^-8.  The reference goes on from the
    block's own normed tokens, logits and choices: a rounding of the tokens changes the
    sign of some up-projections, of a share of about 2^-8, and ReLU's derivative there
    by all of it, which is 2^-4 of the gradient's norm and no error.  Otherwise errors
    add up in the 2-norm: y takes the normed
    tokens', up, y's rows and out (4); the router's weight gradient the normed tokens',
    the logits' (whose error of 2^-8 of a logit of about 1 moves a gate, and what is
    subtracted from one another in its gradient, by as much: 4) and dlogits' (6 in
    all); the norm's gradients those of dx of the experts (8), of the router (8) and
    their sum."""
    ccl()
    torch.manual_seed(0)
    p, T, H, F, E, k = 2, 160, 96, 128, 8, 2
    block, weights = make(p, T, H, F, E, k, score, together)
    x = [torch.randn(T - 7 * r, H, device="cuda").bfloat16() for r in range(p)]
    res = [torch.randn_like(v) for v in x] if residual else None
    y, s, losses = block.forward(x, res)
    held, ends, logits, ids, counts = block.router.saved
    dy, ds = [torch.randn_like(v) for v in x], [torch.randn_like(v) for v in x]
    grads = [[torch.empty_like(w, dtype=torch.float32) for _ in range(p)] for w in weights]
    dx = block.backward(dy, ds, *grads, dlosses=[torch.full((1,), 2.0, device="cuda")] * p, balance_scale=0.5)

    def near(got, want, roundings):
        off, size = float((got.double() - want).norm()), float(want.norm())
        assert off <= roundings * 2.0 ** -8 * size

    total_rows = sum(v.shape[0] for v in x)
    leaves = []
    shares = []
    for r in range(p):
        X, U, D, R, W, B = (t.double().requires_grad_() for t in ((s[r] if residual else x[r]), *weights))
        if residual:
            assert torch.equal(s[r], (x[r].float() + res[r].float()).bfloat16())
        z = (X - X.mean(1, keepdim=True)) / (X.var(1, correction=0, keepdim=True) + 1e-5).sqrt()
        normed = z * W + B
        near(held[r], normed.detach(), 1)
        normed = normed + (held[r].double() - normed).detach()
        l = normed @ R.T
        near(logits[r], l.detach(), 3)
        l = l + (logits[r].double() - l).detach()
        u = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
        chosen = u.gather(1, ids[r].long())
        gates = 1.5 * chosen / chosen.sum(1, keepdim=True)
        hidden = torch.relu(torch.einsum("tkfh,th->tkf", U[ids[r].long()], normed))
        out = torch.einsum("tk,tkhf,tkf->th", gates, D[ids[r].long()], hidden)
        near(y[r], out.detach(), 4)
        share = u / u.sum(1, keepdim=True)
        shares.append(share.sum(0))
        leaves.append((X, U, D, R, W, B, out))
    for r in range(p):
        n = counts[r][:-1].double()
        t = float(total_rows if together else x[r].shape[0])
        assert int(counts[r][-1]) == int(t)
        got = torch.bincount(torch.cat([i.reshape(-1).long() for i in (ids if together else [ids[r]])]), minlength=E)
        assert torch.equal(got, counts[r][:-1].long())
        mine = sum(shares) if together else shares[r]
        loss = E / (k * t * t) * (n * mine).sum()
        near(losses[r], loss.detach()[None], 3)
        X, U, D, R, W, B, out = leaves[r]
        # this rank's part of the one loss, or its own
        own = E / (k * t * t) * (n * shares[r]).sum()
        ((out * dy[r].double()).sum() + (X * ds[r].double()).sum() + 1.0 * own).backward(retain_graph=True)
        near(dx[r], X.grad, 17)
        for g, leaf, roundings in zip(grads, (U, D, R, W, B), (5, 5, 10, 17, 17)):
            near(g[r], leaf.grad, roundings)
    with pytest.raises(RuntimeError, match="without a forward"):
        block.backward(dy, ds, *grads)
    with pytest.raises(RuntimeError, match="without a forward"):
        block.router.backward([], [])


def test_two_blocks_share_the_residual_stream():
    """What the first block hands on is what the second one's norm adds up."""
    ccl()
    torch.manual_seed(1)
    first, _ = make(1, 64, 64, 96, 4, 1, "softmax", False)
    second, _ = make(1, 64, 64, 96, 4, 1, "softmax", False)
    x = [torch.randn(64, 64, device="cuda").bfloat16()]
    y, s, _ = first.forward(x)
    assert s[0] is x[0]
    _, s2, _ = second.forward(y, s)
    assert torch.equal(s2[0], (y[0].float() + x[0].float()).bfloat16())


def test_block_in_a_graph():
    """Forward and backward captured once and replayed on new tokens."""
    ccl()
    torch.manual_seed(2)
    block, weights = make(2, 48, 64, 96, 4, 2, "softmax", True)
    x, res = [torch.randn(48, 64, device="cuda").bfloat16() for _ in range(2)], [torch.randn(48, 64, device="cuda").bfloat16() for _ in range(2)]
    dy, ds = [torch.randn_like(v) for v in x], [torch.randn_like(v) for v in x]
    grads = [[torch.zeros_like(w, dtype=torch.float32) for _ in range(2)] for w in weights]

    def step():
        y, s, losses = block.forward(x, res)
        return y + s + losses + block.backward(dy, ds, *grads, balance_scale=0.1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for v in x + res + dy + ds:
        v.copy_(torch.randn_like(v))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in held] + [t.clone() for g in grads for t in g]
    want = step() + [t for g in grads for t in g]
    for a, b in zip(got, want):
        assert torch.equal(a, b)
