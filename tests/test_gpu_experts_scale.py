"""A rank's own experts where calls are large: more ranks than a launch takes,
as many experts as allowed, weights past 2^32 elements, many tokens of narrow
rows, and the whole way from dispatch to combine."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from a2a_ring_ordered_gb300 import workloads
from gpu_util import ccl
from oracle import experts
from test_gpu_experts import dev, host, rounded

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    return ccl()


# 8 ranks or 2048 (rank, expert) pairs a launch: both limits, and ranks left over
@pytest.mark.parametrize("p,num,n,k", [(19, 5, 72, 40), (5, 1024, 16, 24), (9, 300, 40, 33)])
def test_products_of_more_ranks_than_a_launch_takes(lib, p, num, n, k):
    rng = np.random.default_rng(p)
    counts = [rng.multinomial(0 if r == 2 else 60 + r, np.full(num, 1 / num)) for r in range(p)]
    offsets = [np.concatenate([[0], np.cumsum(c)]).astype(np.int32) for c in counts]
    x, dy = ([rng.integers(-2, 3, (int(o[-1]), width)).astype(np.float32) for o in offsets] for width in (k, n))
    w = rng.integers(-2, 3, (num, n, k)).astype(np.float32)
    d_x, d_dy, d_o, d_w = [dev(v, BF) for v in x], [dev(v, BF) for v in dy], [dev(o) for o in offsets], [dev(w, BF)] * p
    y = [torch.full((v.shape[0], n), 5.0, dtype=BF, device="cuda") for v in x]
    dx = [torch.full((v.shape[0], k), 5.0, dtype=BF, device="cuda") for v in x]
    dw = [torch.full((num, n, k), 5.0, device="cuda") for _ in x]
    before = lib.ccl_kernel_launch_count()
    lib.ccl_moe_product(d_x, d_o, d_w, y)
    assert lib.ccl_kernel_launch_count() - before == -(-p // min(8, 2048 // num))
    lib.ccl_moe_product_grad_input(d_dy, d_o, d_w, dx)
    lib.ccl_moe_product_grad_weight(d_dy, d_x, d_o, dw)
    for r in range(p):
        rows = x[r].shape[0]
        assert torch.equal(y[r].cpu(), rounded(experts.product(x[r], offsets[r], w, np.zeros((rows, n))), BF))
        assert torch.equal(dx[r].cpu(), rounded(experts.product_grad_input(dy[r], offsets[r], w, np.zeros((rows, k))), BF))
        assert torch.equal(dw[r].cpu(), rounded(experts.product_grad_weight(dy[r], x[r], offsets[r]), torch.float32))


def test_weights_past_32_bit_offsets(lib):
    """Two experts of 32768 x 65600: the second one's weights begin past 2^31
    elements and end past 2^32."""
    n, k = 32768, 65600
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randint(-1, 2, (7, k), generator=g, device="cuda").to(BF)
    dy = torch.randint(-1, 2, (7, n), generator=g, device="cuda").to(BF)
    off = torch.tensor([0, 3, 7], dtype=torch.int32, device="cuda")
    dw = torch.empty(2, n, k, dtype=BF, device="cuda")
    lib.ccl_moe_product_grad_weight([dy], [x], [off], [dw])
    for e, (lo, hi) in enumerate(((0, 3), (3, 7))):
        for i in range(0, n, 8192):
            assert torch.equal(dw[e, i:i + 8192].float(), dy[lo:hi, i:i + 8192].float().T @ x[lo:hi].float())
    # the same numbers as weights: at most 4 each, every 64th column of x kept, so
    # that sums of 1025 terms stay whole and below 2^13
    xs = torch.zeros_like(x)
    xs[:, ::64] = x[:, ::64]
    y = torch.empty(7, n, dtype=BF, device="cuda")
    lib.ccl_moe_product([xs], [off], [dw], [y])
    for e, (lo, hi) in enumerate(((0, 3), (3, 7))):
        want = (xs[lo:hi, ::64].double() @ dw[e, :, ::64].double().T).to(BF)
        assert torch.equal(y[lo:hi], want)
    ds = torch.zeros_like(dy)
    ds[:, ::32] = dy[:, ::32]
    dx = torch.empty(7, k, dtype=BF, device="cuda")
    lib.ccl_moe_product_grad_input([ds], [off], [dw], [dx])
    for e, (lo, hi) in enumerate(((0, 3), (3, 7))):
        assert torch.equal(dx[lo:hi], (ds[lo:hi, ::32].double() @ dw[e, ::32].double()).to(BF))


# several passes per CTA, limited by the table of choices (narrow rows, 16 of
# them) or by eight; ranks of other lengths; widths that end inside a pass
@pytest.mark.parametrize("tokens,k,hidden,dtype", [([200000, 7], 16, 64, "bf16"), ([60000, 0, 50001], 3, 200, "bf16"),
                                                   ([90000], 1, 68, "f32"), ([150000, 1], 2, 32, "f32")])
def test_gated_sum_of_many_narrow_rows(lib, tokens, k, hidden, dtype):
    """Against torch in fp32 with the header's order: products and sums rounded one by one."""
    dt = {"f32": torch.float32, "bf16": BF}[dtype]
    g = torch.Generator(device="cuda").manual_seed(k)
    rows, y, w, out = [], [], [], []
    for t in tokens:
        r = torch.randperm(t * k, generator=g, device="cuda").to(torch.int32).view(t, k)
        r[torch.rand(t, k, generator=g, device="cuda") < 0.1] = -1
        rows.append(r)
        y.append(torch.randn(t * k, hidden, generator=g, device="cuda").to(dt))
        w.append(torch.rand(t, k, generator=g, device="cuda"))
        out.append(torch.full((t, hidden), 7.0, device="cuda", dtype=dt))
    lib.ccl_moe_from_experts(y, rows, w, out)
    for r, t in enumerate(tokens):
        acc = torch.zeros(t, hidden, device="cuda")
        for j in range(k):
            at = rows[r][:, j].long()
            term = y[r][at.clamp_min(0)].float() * w[r][:, j:j + 1]
            acc = torch.where((at >= 0)[:, None], acc + term, acc)
        assert torch.equal(out[r], acc.to(dt))


def test_from_dispatch_to_combine(lib):
    """Tokens travel to the ranks that hold their experts, are multiplied there
    and come back: dispatch, sort, rows, products, rows back, combine.  Whole
    numbers: sums below 2^8, so that bf16 holds every intermediate."""
    p, T, k, E, h = 4, 100, 4, 16, 128
    rng = np.random.default_rng(3)
    ids = workloads.moe_topk_routing(p, T, k, E, seed=2)
    x = [rng.integers(-1, 2, (T, h)).astype(np.float32) for _ in range(p)]
    w = np.zeros((E, h, h), np.float32)  # three entries a row: sums of at most 3
    for e in range(E):
        for i in range(h):
            w[e, i, rng.choice(h, 3, replace=False)] = rng.integers(-1, 2, 3)
    gates = [np.full((T, k), 0.5, np.float32) for _ in range(p)]
    d_ids = [dev(i) for i in ids]
    counts = torch.empty(p * p, dtype=torch.int64, device="cuda")
    slots = [torch.empty(T, k, dtype=torch.int32, device="cuda") for _ in range(p)]
    lib.ccl_moe_route(d_ids, E, counts, slots)
    m = counts.cpu().numpy().reshape(p, p).sum(0)
    recv = [torch.empty(int(c), h, dtype=BF, device="cuda") for c in m]
    rexp = [torch.empty(int(c), dtype=torch.int32, device="cuda") for c in m]
    lib.ccl_moe_dispatch([dev(v, BF) for v in x], d_ids, counts, slots, E, recv, None, rexp)
    first = [r * E // p for r in range(p)]
    offsets = [torch.empty(E // p + 1, dtype=torch.int32, device="cuda") for _ in range(p)]
    rows = [torch.empty_like(e) for e in rexp]
    ordered, y, back = ([torch.empty_like(v) for v in recv] for _ in range(3))
    lib.ccl_moe_sort(rexp, E // p, offsets, rows, first_expert=first)
    lib.ccl_moe_to_experts(recv, rows, ordered)
    lib.ccl_moe_product(ordered, offsets, [dev(w[f:f + E // p], BF) for f in first], y)
    lib.ccl_moe_from_experts(y, rows, None, back)
    out = [torch.empty(T, h, dtype=BF, device="cuda") for _ in range(p)]
    lib.ccl_moe_combine(back, d_ids, [dev(v) for v in gates], counts, slots, E, out)
    for r in range(p):
        want = 0.5 * np.einsum("tkij,tj->ti", w[ids[r]], x[r])
        np.testing.assert_array_equal(host(out[r]), want.astype(np.float32))
