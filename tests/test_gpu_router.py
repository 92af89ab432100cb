"""The router's choice, its balance loss and their gradients against the 64-bit definitions.

Tolerances count roundings of 2^-24 (fp32) in the kernels' order of work.  With A the
largest distance of a logit from its row's top: a score is exp of a rounded argument
(A roundings) times a rounded constant (A more), good to two units, sigmoid's quotient
two more: 2 A + 8.  A share or gate is a score over a sum of scores (as far off, and
one rounding for each of its additions, at most E / 8 + 8 in a row), rounded: in all
4 A + E / 8 + 32.  Gradients are sums of products of those with their inputs, each
product as far off; their bound is on the sum of the terms' magnitudes.  A bf16
gradient is rounded once more: 2^-8 / 2 relative to half a step, 2^-9 of the value
above, at most 2^-8 of it.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import GUARD, Guarded, ccl
from oracle import router

pytestmark = pytest.mark.gpu

ONE = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def spread(l: np.ndarray) -> np.ndarray:
    """A of the tolerances, for each row: how far finite logits lie from the row's
    top, and from 0 (sigmoid); what is further than 104 is 0 in fp32."""
    finite = np.isfinite(l)
    top = np.where(finite, l, -np.inf).max(1, initial=-np.inf, keepdims=True)
    far = np.where(finite, np.where(np.isfinite(top), top, 0.0) - np.where(finite, l, 0.0), 0.0)
    size = np.where(finite & (np.abs(l) < 104), np.abs(np.where(finite, l, 0.0)), 0.0)
    return np.maximum(1.0, np.maximum(np.where(far < 104, far, 0.0).max(1, initial=0.0, keepdims=True), size.max(1, initial=0.0, keepdims=True)))


def share_tolerance(l: np.ndarray) -> np.ndarray:
    """For each row."""
    return (4 * spread(l) + l.shape[1] / 8 + 32) * ONE


def make_logits(rng, tokens: int, experts: int, dtype: str, ties: bool = True, masked: bool = True) -> np.ndarray:
    l = rng.normal(size=(tokens, experts)) * 2
    if ties:
        l[: tokens // 2] = np.round(l[: tokens // 2])  # many equal ones
    if masked and experts > 2:
        l[:, experts // 2] = -np.inf
        l[tokens // 3] = -np.inf  # nothing left
        l[tokens // 4, 1:] = -np.inf  # one left
        l[-1] = torch.finfo(DT[dtype]).min  # a mask by the type's lowest value: all alike
    return torch.tensor(l).to(DT[dtype]).double().numpy()


class Buffer(Guarded):
    """Guarded, of a shape; `off`: one element off the 16-byte grid."""

    def __init__(self, shape, dtype: str, off: bool = False, value: np.ndarray | None = None):
        super().__init__(int(np.prod(shape)), dtype, GUARD + 1 if off else GUARD)
        self.t = self.view.view(*shape)
        if value is not None:
            self.t.copy_(torch.tensor(value).to(self.t.dtype))

    def numpy(self) -> np.ndarray:
        assert self.guards_intact()
        return self.t.double().cpu().numpy() if self.t.is_floating_point() else self.t.cpu().numpy()


SHAPES = [  # tokens of each rank, experts, k
    ([1], 1, 1), ([1], 2, 2), ([5, 0, 3], 4, 2), ([33, 7], 8, 2), ([64], 16, 16), ([1], 32, 4), ([40, 1], 33, 3), ([257], 60, 6),
    ([12], 61, 8), ([100, 31, 64, 1], 64, 8), ([77], 128, 8), ([50, 9], 160, 6), ([1], 256, 8), ([130, 300], 256, 8), ([19], 257, 4),
    ([21], 384, 8), ([10], 512, 1), ([9, 2], 1000, 16), ([17], 1024, 12),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,experts,k", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_gate_and_balance(tokens, experts, k, dtype, score):
    c = ccl()
    rng = np.random.default_rng(experts * 31 + k)
    for off, normalize, scale, together in ((False, True, 1.0, False), (True, False, 2.5, True)):
        logits = [make_logits(rng, t, experts, dtype) if t else np.zeros((0, experts)) for t in tokens]
        l = [Buffer(v.shape, dtype, off, v) for v in logits]
        ids, gates = [Buffer((t, k), "i32") for t in tokens], [Buffer((t, k), "f32") for t in tokens]
        counts, losses = [Buffer((experts + 1,), "i32") for _ in tokens], [Buffer((1,), "f32") for _ in tokens]
        args = ([b.t for b in l], [b.t for b in ids], [b.t for b in gates])
        c.ccl_moe_gate(*args, score=score, normalize=normalize, scale=scale)
        alone = [(b.numpy().copy(), g.numpy().copy()) for b, g in zip(ids, gates)]
        c.ccl_moe_gate(*args, score=score, normalize=normalize, scale=scale, counts=[b.t for b in counts], losses=[b.t for b in losses],
                       together=together)
        want = [router.choose(v, k) for v in logits]
        n = [router.counts(v, i) for v, i in zip(logits, want)]
        if together:
            n = [sum(n)] * len(n)
        for r, v in enumerate(logits):
            np.testing.assert_array_equal(ids[r].numpy(), want[r])
            np.testing.assert_array_equal(alone[r][0], want[r])
            np.testing.assert_array_equal(alone[r][1], gates[r].numpy())
            g = router.gates(v, want[r], score, normalize, scale)
            assert (np.abs(gates[r].numpy() - g) <= share_tolerance(v) * g + 1e-38).all()
            np.testing.assert_array_equal(counts[r].numpy(), n[r])
        check_losses(losses, logits, n, k, score, together)
        # the loss alone, of these ids
        again_n, again = [Buffer((experts + 1,), "i32") for _ in tokens], [Buffer((1,), "f32") for _ in tokens]
        c.ccl_moe_balance([b.t for b in l], [b.t for b in ids], [b.t for b in again_n], [b.t for b in again], score=score, together=together)
        for r in range(len(tokens)):
            np.testing.assert_array_equal(again_n[r].numpy(), n[r])
        check_losses(again, logits, n, k, score, together)


def check_losses(losses, logits, n, k, score, together):
    """Shares are positive: a loss is as far off as they are, and by the additions
    over the rows that a warp has, one rounding each."""
    for r, v in enumerate(logits):
        mine = [x for x in logits if x.size] if together else [v]
        want = router.balance_loss(mine, n[r], k, score) if n[r][-1] else 0.0
        rows = max(x.shape[0] for x in logits)
        tol = max((share_tolerance(x).max() for x in mine if x.size), default=0.0) + (rows + 8) * ONE
        assert abs(losses[r].numpy()[0] - want) <= tol * want


def grad_terms(l, ids, d, score, normalize, scale, n, k, dloss):
    """(gradient, sum of its terms' magnitudes)."""
    out, size = np.zeros_like(l), np.zeros_like(l)
    p = router.shares(l, score)
    away = 1.0 if score == "softmax" else router._sigmoid(-l)
    if d is not None:
        out += router.gate_grad(l, ids, d, score, normalize, scale)
        there = (ids >= 0) & (ids < l.shape[1])
        g, m = router.gates(l, ids, score, normalize, scale), np.where(there, np.abs(d), 0.0)
        mean = (g * m).sum(1, keepdims=True) / scale
        own = g * (m + mean)
        for t in range(l.shape[0]):
            np.add.at(size[t], np.where(there, ids, 0)[t], np.where(there, own, 0.0)[t])
        if not normalize:
            size += p * (g * m).sum(1, keepdims=True)
    if n is not None:
        out += router.balance_grad(l, n, k, score, dloss)
        a = np.abs(n[:-1] - n[:-1].mean()) * abs(dloss) * l.shape[1] / (k * max(1.0, float(n[-1])) ** 2)
        size += p * (a + (p * a).sum(1, keepdims=True))
    return out, size * away


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,experts,k", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_gradients(tokens, experts, k, dtype, score):
    c = ccl()
    rng = np.random.default_rng(experts * 17 + k)
    for off, normalize, scale, kind in ((False, True, 1.0, "gates"), (True, False, 2.5, "gates"), (False, False, 1.0, "both"), (True, True, 2.5, "both"),
                                        (False, None, None, "balance"), (True, None, None, "balance")):
        logits = [make_logits(rng, t, experts, dtype) if t else np.zeros((0, experts)) for t in tokens]
        chosen = [router.choose(v, k) for v in logits]
        n = [router.counts(v, i) for v, i in zip(logits, chosen)]
        for v in chosen:
            if v.size and k > 1:
                v[0, 1] = v[0, 0]  # an expert twice
                v[-1, 0] = experts  # none of the experts
        d = [rng.normal(size=v.shape).astype(np.float32) for v in chosen]
        for v, x in zip(chosen, d):
            x[v < 0] = np.nan  # nothing is read beside a choice that is none
        dloss = [np.float32(rng.normal()) for _ in tokens]
        l = [Buffer(v.shape, dtype, off, v) for v in logits]
        ids, dgates = [Buffer(v.shape, "i32", False, v) for v in chosen], [Buffer(v.shape, "f32", False, v) for v in d]
        counts, dlosses = [Buffer(v.shape, "i32", False, v) for v in n], [Buffer((1,), "f32", False, np.array([v])) for v in dloss]
        out = [Buffer(v.shape, dtype, off) for v in logits]
        lists = [[b.t for b in bs] for bs in (l, ids, dgates, out, counts, dlosses)]
        if kind == "balance":
            c.ccl_moe_balance_grad(lists[0], lists[4], lists[3], k, score=score, dlosses=lists[5], scale=0.5)
        else:
            more = dict(counts=lists[4], dlosses=lists[5], balance_scale=0.5) if kind == "both" else {}
            c.ccl_moe_gate_grad(*lists[:4], score=score, normalize=normalize, scale=scale, **more)
        for r, v in enumerate(logits):
            if not v.size:
                continue
            want, size = grad_terms(v, chosen[r], None if kind == "balance" else d[r], score, normalize, scale,
                                    None if kind == "gates" else n[r], k, 0.5 * float(dloss[r]))
            got = out[r].numpy()
            assert np.isfinite(got).all()
            step = 2.0 ** -8 if dtype == "bf16" else ONE
            assert (np.abs(got - want) <= 2 * share_tolerance(v) * size + step * np.abs(want) + 1e-38).all()


@pytest.mark.parametrize("experts,k", [(8, 3), (60, 6), (256, 8), (256, 16), (300, 8), (1024, 16)])
def test_choice_by_the_last_bit(experts, k):
    """fp32 logits that differ in their last bits alone, around 0 too."""
    c = ccl()
    rng = np.random.default_rng(experts + k)
    v = (1.0 + rng.integers(-300, 300, size=(90, experts)) * 2.0 ** -23).astype(np.float32)
    v[30:60] = (rng.integers(-5, 5, size=(30, experts)) * 2.0 ** -149).astype(np.float32)
    v[60:, ::2] *= -1
    ids, gates = [torch.empty(90, k, dtype=torch.int32, device="cuda")], [torch.empty(90, k, device="cuda")]
    c.ccl_moe_gate([torch.from_numpy(v).cuda()], ids, gates)
    np.testing.assert_array_equal(ids[0].cpu().numpy(), router.choose(v, k))


def test_gates_of_chosen_experts_far_below_the_row():
    """Given ids whose logits are far below the row's largest still share their gates."""
    c = ccl()
    l = torch.zeros(5, 16, device="cuda")
    l[:, 0] = 300.0
    ids, d = [torch.tensor([[1, 2]] * 5, dtype=torch.int32, device="cuda")], [torch.tensor([[1.0, -1.0]] * 5, device="cuda")]
    for score in ("softmax", "sigmoid"):
        out = [torch.empty_like(l)]
        c.ccl_moe_gate_grad([l], ids, d, out, score=score)
        want = router.gate_grad(l.double().cpu().numpy(), ids[0].cpu().numpy(), d[0].cpu().numpy(), score, True, 1.0)
        if score == "softmax":  # the 64-bit definition keeps the row's largest: exp(-300) is a number there
            assert want[0, 1] == 0.5
        np.testing.assert_allclose(out[0].cpu().numpy(), want, rtol=64 * ONE, atol=0)


def test_without_dlosses_they_are_ones():
    c = ccl()
    l = [torch.randn(50, 16, device="cuda")]
    counts = [torch.randint(0, 20, (17,), dtype=torch.int32, device="cuda")]
    a, b = [torch.empty_like(l[0])], [torch.empty_like(l[0])]
    c.ccl_moe_balance_grad(l, counts, a, 2, scale=0.25)
    c.ccl_moe_balance_grad(l, counts, b, 2, dlosses=[torch.full((1,), 0.25, device="cuda")])
    assert torch.equal(a[0], b[0]) and a[0].abs().max() > 0


def test_one_expert_left_gets_no_gradient():
    """Its share is 1 whatever its logit: the gradients are 0 to the bit."""
    c = ccl()
    l = torch.full((40, 24), -float("inf"), device="cuda")
    l[torch.arange(40), torch.arange(40) % 24] = torch.randn(40, device="cuda") * 30
    ids, gates = [torch.empty(40, 3, dtype=torch.int32, device="cuda")], [torch.empty(40, 3, device="cuda")]
    counts, losses = [torch.empty(25, dtype=torch.int32, device="cuda")], [torch.empty(1, device="cuda")]
    for score in ("softmax", "sigmoid"):
        c.ccl_moe_gate([l], ids, gates, score=score, counts=counts, losses=losses)
        assert (gates[0][:, 0] == 1).all() and (gates[0][:, 1:] == 0).all()
        assert (ids[0][:, 0] == torch.arange(40, device="cuda") % 24).all() and (ids[0][:, 1:] == -1).all()
        out = [torch.empty_like(l)]
        c.ccl_moe_balance_grad([l], counts, out, 3, score=score)
        assert (out[0] == 0).all()
        for normalize in (True, False) if score == "softmax" else (True,):
            c.ccl_moe_gate_grad([l], ids, [torch.randn(40, 3, device="cuda")], out, score=score, normalize=normalize)
            assert (out[0] == 0).all()
            c.ccl_moe_gate_grad([l], ids, [torch.randn(40, 3, device="cuda")], out, score=score, normalize=normalize, counts=counts)
            assert (out[0] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts", [8, 60, 256, 1000])
def test_nan_and_infinities_choose_in_bounds(dtype, experts):
    """NaN comes first, +inf next; ids stay in range and other rows keep their values."""
    c = ccl()
    rng = np.random.default_rng(experts)
    v = make_logits(rng, 40, experts, dtype)
    v[3, 5], v[4, 6], v[4, 2], v[5] = np.nan, np.nan, np.inf, np.inf
    l = [Buffer(v.shape, dtype, False, v)]
    ids, gates = [Buffer((40, 4), "i32")], [Buffer((40, 4), "f32")]
    c.ccl_moe_gate([l[0].t], [ids[0].t], [gates[0].t])
    np.testing.assert_array_equal(ids[0].numpy(), router.choose(v, 4))
    got = gates[0].numpy()
    assert np.isnan(got[3, 0]) and np.isnan(got[4, 0])
    rest = [t for t in range(40) if t not in (3, 4, 5)]
    want = router.gates(v[rest], ids[0].numpy()[rest], "softmax", True, 1.0)
    assert (np.abs(got[rest] - want) <= share_tolerance(v[rest]) * want).all()


def test_same_bits_whatever_the_workspace_held_and_in_a_graph():
    c = ccl()
    torch.manual_seed(0)
    p, T, E, k = 3, 1001, 96, 6
    l = [torch.randn(T + r, E, device="cuda").bfloat16() for r in range(p)]
    ids = [torch.empty(T + r, k, dtype=torch.int32, device="cuda") for r in range(p)]
    gates = [torch.empty(T + r, k, device="cuda") for r in range(p)]
    counts, losses = [torch.empty(E + 1, dtype=torch.int32, device="cuda") for _ in range(p)], [torch.empty(1, device="cuda") for _ in range(p)]
    ws = torch.full((c.ccl_moe_balance_workspace_bytes(p, E),), 0xFF, dtype=torch.uint8, device="cuda")
    alone = [torch.empty_like(t) for t in counts], [torch.empty_like(t) for t in losses]
    outs = ids + gates + counts + losses + alone[0] + alone[1]

    def both(**kw):
        c.ccl_moe_gate(l, ids, gates, counts=counts, losses=losses, **kw)
        c.ccl_moe_balance(l, ids, *alone)

    both(workspace=ws)
    first = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for t in outs:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, outs):
        assert torch.equal(a, b)


def test_two_streams_with_workspaces_of_their_own():
    c = ccl()
    torch.manual_seed(1)
    E, k = 64, 4
    l = [torch.randn(20000, E, device="cuda") for _ in range(2)]
    out = []
    for v in l:
        ids, gates = [torch.empty(20000, k, dtype=torch.int32, device="cuda")], [torch.empty(20000, k, device="cuda")]
        out.append((ids, gates, [torch.empty(E + 1, dtype=torch.int32, device="cuda")], [torch.empty(1, device="cuda")]))
    want = []
    for v, (ids, gates, n, loss) in zip(l, out):
        c.ccl_moe_gate([v], ids, gates, counts=n, losses=loss)
        want.append([t.clone() for t in (ids[0], gates[0], n[0], loss[0])])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in l]
    for _ in range(5):
        for s, v, (ids, gates, n, loss) in zip(streams, l, out):
            c.ccl_moe_gate([v], ids, gates, counts=n, losses=loss, stream=s)
    torch.cuda.synchronize()
    for w, (ids, gates, n, loss) in zip(want, out):
        for a, b in zip(w, (ids[0], gates[0], n[0], loss[0])):
            assert torch.equal(a, b)


def test_refusals():
    c = ccl()
    l = [torch.randn(4, 8, device="cuda")]
    ids, gates = [torch.empty(4, 2, dtype=torch.int32, device="cuda")], [torch.empty(4, 2, device="cuda")]
    with pytest.raises(ValueError, match="score"):
        c.ccl_moe_gate(l, ids, gates, score="tanh")
    with pytest.raises(ValueError, match="a row per token"):
        c.ccl_moe_gate(l, [torch.empty(3, 2, dtype=torch.int32, device="cuda")], gates)
    with pytest.raises(ValueError, match="given together"):
        c.ccl_moe_gate(l, ids, gates, counts=[torch.empty(9, dtype=torch.int32, device="cuda")])
    with pytest.raises(c.CclError, match="k=9 of 8"):
        c.ccl_moe_gate(l, [torch.empty(4, 9, dtype=torch.int32, device="cuda")], [torch.empty(4, 9, device="cuda")])
    with pytest.raises(c.CclError, match="fp32 or bf16"):
        c.ccl_moe_gate([torch.zeros(4, 8, dtype=torch.int32, device="cuda")], ids, gates)
    with pytest.raises(ValueError, match="unsupported dtype"):
        c.ccl_moe_gate([torch.zeros(4, 8, dtype=torch.float16, device="cuda")], ids, gates)
    with pytest.raises(ValueError, match="contiguous"):
        c.ccl_moe_gate([torch.randn(8, 4, device="cuda").t()], ids, gates)
    n, loss = [torch.empty(9, dtype=torch.int32, device="cuda")], [torch.empty(1, device="cuda")]
    with pytest.raises(c.CclError, match="workspace"):
        c.ccl_moe_balance(l, ids, n, loss, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(c.CclError, match="dlosses needs counts"):
        c.ccl_moe_gate_grad(l, ids, gates, [torch.empty_like(l[0])], dlosses=loss)
    with pytest.raises(c.CclError, match="overlaps"):
        c.ccl_moe_gate_grad(l, ids, gates, l)
    with pytest.raises(c.CclError, match="scale"):
        c.ccl_moe_gate(l, ids, gates, scale=float("nan"))
