"""GPU parity of a rank's own experts: sort, rows, products and their gradients.

Tolerances.  u = 2^-24 is fp32's rounding unit, 2^-8 bf16's.  A sum of n fp32
products, each rounded, is within (n + 1) * 2^-23 of the sum of the products'
magnitudes in any order (the classic bound with u doubled for the second-order
terms); writing bf16 adds 2^-8 of the value.  The tensor cores' products of
bf16 numbers are exact, their sums cut rather than rounded at the accumulator's
last bit: the same bound holds with u doubled, which 2^-23 already is.  Whole
numbers small enough are exact all through and are compared bit by bit.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from a2a_ring_ordered_gb300 import workloads
from gpu_util import ccl
from oracle import experts

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def lib():
    return ccl()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def bf16_exact(rng, shape, scale=1.0):
    """Random values that bf16 holds exactly, as fp32."""
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16().float().numpy()


def shifted(a, dtype, off):
    """A contiguous device tensor with a's values that starts `off` elements into its storage."""
    store = torch.zeros(a.size + off + 8, dtype=dtype, device="cuda")
    view = store[off:off + a.size].view(a.shape)
    view.copy_(torch.from_numpy(np.ascontiguousarray(a)))
    return view


def ids_of(rng, tokens, k, num, skew=1.0):
    """Distinct experts per token, popular ones first."""
    if tokens == 0:
        return np.zeros((0, k), dtype=np.int32)
    g = rng.gumbel(size=(tokens, num)) - skew * np.log(np.arange(num) + 1.0)
    return np.argsort(-g, axis=1)[:, :k].astype(np.int32)


# ------------------------------------------------------------------- sort
def run_sort(lib, ids, num, first=None):
    p = len(ids)
    d = [dev(i) for i in ids]
    offsets = [torch.full((num + 1,), -9, dtype=torch.int32, device="cuda") for _ in range(p)]
    rows = [torch.full_like(i, -9) for i in d]
    lib.ccl_moe_sort(d, num, offsets, rows, first_expert=first)
    return offsets, rows


# one item; less than a warp; one CTA; several CTAs; a rank with nothing; as
# many experts as allowed; every item of one expert
@pytest.mark.parametrize("tokens,k,num", [([1], 1, 1), ([3], 8, 256), ([40, 0, 7], 3, 5), ([5000], 8, 64),
                                          ([513, 2049], 2, 1024), ([200000], 1, 8), ([70000, 30], 4, 33)])
def test_sort(lib, tokens, k, num):
    rng = np.random.default_rng(num)
    ids = [ids_of(rng, t, k, max(num, k))[:, :k] for t in tokens]
    offsets, rows = run_sort(lib, ids, num)
    for r, i in enumerate(ids):
        want = experts.sort(i, num)
        np.testing.assert_array_equal(host(offsets[r]), want[0])
        np.testing.assert_array_equal(host(rows[r]), want[1])


def test_sort_one_expert_and_strangers(lib):
    ids = [np.full((3000, 2), 4, np.int32), np.array([[-1, 2 ** 31 - 1], [-2 ** 31, 3], [7, 8]], np.int32)]
    offsets, rows = run_sort(lib, ids, 4, first=[4, 5])
    assert host(offsets[0]).tolist() == [0, 6000, 6000, 6000, 6000]
    assert (host(rows[0]).reshape(-1) == np.arange(6000)).all()
    assert host(offsets[1]).tolist() == [0, 0, 0, 1, 2]
    assert host(rows[1]).tolist() == [[-1, -1], [-1, -1], [0, 1]]


def test_sort_follows_dispatch(lib):
    """recv_expert of a dispatch, with k = 1 and the rank's first expert: the local order."""
    p, T, k, E, h = 4, 300, 4, 16, 128
    ids = workloads.moe_topk_routing(p, T, k, E, seed=1)
    d_ids = [dev(i) for i in ids]
    counts = torch.empty(p * p, dtype=torch.int64, device="cuda")
    slots = [torch.empty(T, k, dtype=torch.int32, device="cuda") for _ in range(p)]
    lib.ccl_moe_route(d_ids, E, counts, slots)
    n = counts.cpu().numpy().reshape(p, p).sum(0)
    x = [torch.randn(T, h, device="cuda").bfloat16() for _ in range(p)]
    recv = [torch.empty(int(m), h, dtype=torch.bfloat16, device="cuda") for m in n]
    rexp = [torch.empty(int(m), dtype=torch.int32, device="cuda") for m in n]
    lib.ccl_moe_dispatch(x, d_ids, counts, slots, E, recv, None, rexp)
    first = [r * E // p for r in range(p)]
    offsets = [torch.empty(E // p + 1, dtype=torch.int32, device="cuda") for _ in range(p)]
    rows = [torch.empty_like(e) for e in rexp]
    ordered = [torch.empty_like(v) for v in recv]
    back = [torch.empty_like(v) for v in recv]
    lib.ccl_moe_sort(rexp, E // p, offsets, rows, first_expert=first)
    lib.ccl_moe_to_experts(recv, rows, ordered)
    lib.ccl_moe_from_experts(ordered, rows, None, back)
    for r in range(p):
        want = experts.sort(host(rexp[r])[:, None], E // p, first[r])
        np.testing.assert_array_equal(host(offsets[r]), want[0])
        assert (host(rexp[r])[np.argsort(host(rows[r]))] == np.sort(host(rexp[r]))).all()
        assert torch.equal(back[r], recv[r])


# -------------------------------------------------------------------- rows
ROWS = [  # tokens of each rank, k, experts (of), hidden, element offset of the buffers
    ([1], 1, 1, 1, 0), ([3], 2, 4, 7, 0), ([64], 8, 256, 4096, 0), ([33, 5, 0], 4, 8, 384, 0), ([17], 16, 40, 1001, 0),
    ([50], 3, 9, 256, 1), ([9], 9, 12, 7168, 0), ([300, 2], 1, 6, 130, 0), ([20], 6, 10, 64, 4), ([31], 2, 5, 63, 3),
]


def make_rows(lib, tokens, k, of, seed, share=1.0):
    """rows of a sort whose rank holds the first `share` of the experts."""
    rng = np.random.default_rng(seed)
    ids = [ids_of(rng, t, k, max(of, k)) for t in tokens]
    num = max(1, int(max(of, k) * share))
    return rng, [experts.sort(i, num)[1] for i in ids]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("share", [1.0, 0.5])
@pytest.mark.parametrize("tokens,k,of,hidden,off", ROWS)
def test_to_experts(lib, tokens, k, of, hidden, off, share, dtype):
    rng, rows = make_rows(lib, tokens, k, of, hidden, share)
    x = [bf16_exact(rng, (t, hidden)) for t in tokens]
    cap = [t * k - (t * k > 5) for t in tokens]  # the last row may not fit
    into = [np.full((c, hidden), 3.0, np.float32) for c in cap]
    out = [shifted(i, DT[dtype], off) for i in into]
    lib.ccl_moe_to_experts([shifted(v, DT[dtype], off) for v in x], [dev(r) for r in rows], out)
    for r in range(len(tokens)):
        np.testing.assert_array_equal(host(out[r]), experts.to_experts(x[r], rows[r], into[r]))
        store = out[r]._base if out[r]._base is not None else out[r]
        flat = store.reshape(-1)
        assert (flat[:off] == 0).all() and (flat[off + cap[r] * hidden:] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("share", [1.0, 0.3])
@pytest.mark.parametrize("tokens,k,of,hidden,off", ROWS)
def test_from_experts_and_its_gradient(lib, tokens, k, of, hidden, off, share, gated, dtype):
    rng, rows = make_rows(lib, tokens, k, of, hidden + 1, share)
    cap = [t * k - (t * k > 5) for t in tokens]
    y = [bf16_exact(rng, (c, hidden)) for c in cap]
    dout = [bf16_exact(rng, (t, hidden)) for t in tokens]
    w = [rng.standard_normal((t, k)).astype(np.float32) for t in tokens]
    dw_ = [dev(v) for v in w] if gated else None
    d_rows, d_y = [dev(r) for r in rows], [shifted(v, DT[dtype], off) for v in y]
    out = [shifted(np.full((t, hidden), 7.0, np.float32), DT[dtype], off) for t in tokens]
    lib.ccl_moe_from_experts(d_y, d_rows, dw_, out)
    dy = [shifted(np.full((c, hidden), 3.0, np.float32), DT[dtype], off) for c in cap]
    dweights = [torch.full((t, k), 9.0, device="cuda") for t in tokens]
    d_dout = [shifted(v, DT[dtype], off) for v in dout]
    lib.ccl_moe_from_experts_grad(d_dout, d_y, d_rows, dw_, dy, dweights)
    only = [shifted(np.full((c, hidden), 3.0, np.float32), DT[dtype], off) for c in cap]
    lib.ccl_moe_from_experts_grad(d_dout, None, d_rows, dw_, only, None)
    only_w = [torch.full((t, k), 9.0, device="cuda") for t in tokens]
    lib.ccl_moe_from_experts_grad(d_dout, d_y, d_rows, dw_, None, only_w)
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    for r, t in enumerate(tokens):
        gate = w[r] if gated else None
        want, size = experts.from_experts(y[r], rows[r], gate)
        assert (np.abs(host(out[r]) - want) <= (k + 1) * 2.0 ** -23 * size + half * np.abs(want) * 1.001).all()
        want_dy, want_dw, size = experts.from_experts_grad(dout[r], y[r], rows[r], gate, np.full((cap[r], hidden), 3.0))
        assert (np.abs(host(dy[r]) - want_dy) <= (2.0 ** -24 + half * 1.001) * np.abs(want_dy)).all()
        assert (np.abs(host(dweights[r]) - want_dw) <= (hidden + 1) * 2.0 ** -23 * size).all()
        assert torch.equal(only[r], dy[r]) and torch.equal(only_w[r], dweights[r])


def test_from_experts_is_deterministic_and_ordered(lib):
    """fp32 terms 2^24, 1, 1, -2^24 in choice order: each sum is rounded before the next."""
    y = np.array([[2.0 ** 24], [1.0], [1.0], [-2.0 ** 24]], np.float32)
    out = [torch.empty(1, 1, device="cuda")]
    lib.ccl_moe_from_experts([dev(y)], [dev(np.array([[0, 1, 2, 3]], np.int32))], None, out)
    assert out[0].item() == 0.0
    lib.ccl_moe_from_experts([dev(y)], [dev(np.array([[1, 2, 0, 3]], np.int32))], None, out)
    assert out[0].item() == 2.0


def test_rows_without_a_choice_do_not_touch_values_that_are_not_finite(lib):
    """A dropped choice reads nothing: NaN in row 0 stays away from it."""
    y = [torch.full((4, 64), float("nan"), device="cuda")]
    rows = [torch.tensor([[-1, -1], [-1, 4], [2 ** 31 - 1, -5]], dtype=torch.int32, device="cuda")]
    out = [torch.full((3, 64), 5.0, device="cuda")]
    dw = [torch.full((3, 2), 5.0, device="cuda")]
    lib.ccl_moe_from_experts(y, rows, [torch.full((3, 2), float("inf"), device="cuda")], out)
    lib.ccl_moe_from_experts_grad(out, y, rows, None, None, dw)
    assert (out[0] == 0).all() and (dw[0] == 0).all()


def test_gates_gradient_against_differences(lib):
    """<from_experts(y, w), g> is linear in each gate: its difference quotient
    over a step of 1 is the gradient.  fp32 outputs carry (k + 1) * 2^-23 of
    their terms' magnitudes each, summed over the row."""
    rng, rows = make_rows(lib, [6], 3, 5, 2)
    h = 40
    y, g = rng.standard_normal((18, h)).astype(np.float32), rng.standard_normal((6, h)).astype(np.float32)
    w = rng.random((6, 3)).astype(np.float32)
    dw, out = [torch.empty(6, 3, device="cuda")], [torch.empty(6, h, device="cuda")]
    lib.ccl_moe_from_experts_grad([dev(g)], [dev(y)], [dev(rows[0])], [dev(w)], None, dw)

    def total(weights):
        lib.ccl_moe_from_experts([dev(y)], [dev(rows[0])], [dev(weights)], out)
        return (host(out[0]).astype(np.float64) * g).sum()

    for t, j in np.ndindex(w.shape):
        up, down = w.copy(), w.copy()
        up[t, j] += 1
        down[t, j] -= 1
        step = np.float64(up[t, j]) - np.float64(down[t, j])
        size = (experts.from_experts(y, rows[0], np.abs(up) + 1)[1] * np.abs(g)).sum()
        slack = 2 * 4 * 2.0 ** -23 * size
        assert abs((total(up) - total(down)) / step - host(dw[0])[t, j]) <= slack


# ---------------------------------------------------------------- products
# rows per expert, n, contract: tiles of one, ragged ones, empty experts at the
# ends and between, single rows, widths off every grid, deep and wide
PRODUCTS = [([1], 1, 1), ([0, 3, 0], 8, 16), ([5, 0, 130, 1, 64], 72, 200), ([128, 128], 128, 128), ([300], 264, 520),
            ([7, 250, 33, 0], 77, 131), ([129, 1, 127], 384, 64), ([17] * 9, 136, 1032), ([0, 0], 64, 64),
            ([1] * 40, 256, 512), ([1000, 24], 512, 256), ([2, 515], 1024, 2056), ([64, 200], 130, 66),
            ([1400, 70, 1000, 3, 641, 129], 1288, 1544), ([833, 65, 1090], 1281, 1403)]


def product_inputs(rng, counts, n, k, whole):
    rows, e = sum(counts), len(counts)
    if whole:
        a, w, d = (rng.integers(-3, 4, s).astype(np.float32) for s in ((rows, k), (e, n, k), (rows, n)))
    else:
        a, w, d = bf16_exact(rng, (rows, k)), bf16_exact(rng, (e, n, k), k ** -0.5), bf16_exact(rng, (rows, n))
    return a, w, d, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def near(got, want, size, depth, dtype):
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    bound = (depth + 1) * 2.0 ** -23 * size + half * np.abs(want) * 1.001
    assert (np.abs(host(got) - want) <= bound + 1e-37).all(), float(np.max(np.abs(host(got) - want) - bound))


def rounded(want, dtype):
    return torch.from_numpy(want).float().to(dtype)


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("off", [0, 1, 4])
@pytest.mark.parametrize("counts,n,k", PRODUCTS)
def test_product(lib, counts, n, k, off, whole):
    rng = np.random.default_rng(n + k)
    x, w, _, offsets = product_inputs(rng, counts, n, k, whole)
    y = shifted(np.full((x.shape[0], n), 5.0, np.float32), torch.bfloat16, off)
    lib.ccl_moe_product([shifted(x, torch.bfloat16, off)], [dev(offsets)], [shifted(w, torch.bfloat16, off)], [y])
    want = experts.product(x, offsets, w, np.zeros((x.shape[0], n)))
    if whole:
        assert torch.equal(y.cpu(), rounded(want, torch.bfloat16))
    else:
        near(y, want, experts.product(np.abs(x), offsets, np.abs(w), np.zeros_like(want)), k, torch.bfloat16)
    store = y._base.reshape(-1)
    assert (store[:off] == 0).all() and (store[off + y.numel():] == 0).all()


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("off", [0, 1, 4])
@pytest.mark.parametrize("counts,n,k", PRODUCTS)
def test_product_grad_input(lib, counts, n, k, off, whole):
    rng = np.random.default_rng(n + k + 1)
    _, w, dy, offsets = product_inputs(rng, counts, n, k, whole)
    dx = shifted(np.full((dy.shape[0], k), 5.0, np.float32), torch.bfloat16, off)
    lib.ccl_moe_product_grad_input([shifted(dy, torch.bfloat16, off)], [dev(offsets)],
                                   [shifted(w, torch.bfloat16, off)], [dx])
    want = experts.product_grad_input(dy, offsets, w, np.zeros((dy.shape[0], k)))
    if whole:
        assert torch.equal(dx.cpu(), rounded(want, torch.bfloat16))
    else:
        near(dx, want, experts.product_grad_input(np.abs(dy), offsets, np.abs(w), np.zeros_like(want)), n, torch.bfloat16)
    store = dx._base.reshape(-1)
    assert (store[:off] == 0).all() and (store[off + dx.numel():] == 0).all()


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("off", [0, 1, 4])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts,n,k", PRODUCTS)
def test_product_grad_weight(lib, counts, n, k, off, dtype, whole):
    rng = np.random.default_rng(n + k + 2)
    x, w, dy, offsets = product_inputs(rng, counts, n, k, whole)
    dw = shifted(np.full(w.shape, 5.0, np.float32), DT[dtype], off)
    lib.ccl_moe_product_grad_weight([shifted(dy, torch.bfloat16, off)], [shifted(x, torch.bfloat16, off)],
                                    [dev(offsets)], [dw])
    want = experts.product_grad_weight(dy, x, offsets)
    if whole:
        assert torch.equal(dw.cpu(), rounded(want, DT[dtype]))
    else:
        near(dw, want, experts.product_grad_weight(np.abs(dy), np.abs(x), offsets), max(counts), DT[dtype])
    store = dw._base.reshape(-1)
    assert (store[:off] == 0).all() and (store[off + dw.numel():] == 0).all()


def test_product_ranks_share_weights_and_skip_foreign_rows(lib):
    """Two ranks with other counts and one set of weights; rows before the first
    offset and after the last belong to nobody: they are neither read into a
    result (they hold NaN) nor written."""
    rng = np.random.default_rng(5)
    n, k = 136, 96
    w = dev(rng.integers(-3, 4, (3, n, k)).astype(np.float32), torch.bfloat16)
    offsets = [np.array([2, 40, 40, 171], np.int32), np.array([0, 1, 5, 9], np.int32)]
    x, y, dx, dw = [], [], [], []
    for o, rows in zip(offsets, (180, 9)):
        v = rng.integers(-3, 4, (rows, k)).astype(np.float32)
        v[:o[0]], v[o[-1]:] = np.nan, np.nan
        x.append(v)
        y.append(torch.full((rows, n), 5.0, device="cuda").bfloat16())
        dx.append(torch.full((rows, k), 5.0, device="cuda").bfloat16())
        dw.append(torch.full((3, n, k), 5.0, device="cuda"))
    d_x, d_o = [dev(v, torch.bfloat16) for v in x], [dev(o) for o in offsets]
    lib.ccl_moe_product(d_x, d_o, [w, w], y)
    d = [np.where(np.isnan(v[:, :1]), np.nan, rng.integers(-3, 4, (v.shape[0], n))).astype(np.float32) for v in x]
    d_d = [dev(v, torch.bfloat16) for v in d]
    lib.ccl_moe_product_grad_input(d_d, d_o, [w, w], dx)
    lib.ccl_moe_product_grad_weight(d_d, d_x, d_o, dw)
    for r, o in enumerate(offsets):
        rows = x[r].shape[0]
        five = np.full((rows, n), 5.0)
        assert torch.equal(y[r].cpu(), rounded(experts.product(x[r], o, host(w), five), torch.bfloat16))
        five = np.full((rows, k), 5.0)
        assert torch.equal(dx[r].cpu(), rounded(experts.product_grad_input(d[r], o, host(w), five), torch.bfloat16))
        assert torch.equal(dw[r].cpu(), rounded(experts.product_grad_weight(d[r], x[r], o), torch.float32))


def test_product_gradients_against_differences(lib):
    """<product(x, w), g> is linear in x and in w: the difference over a step of
    2 in one whole-number input is exact (every sum stays below 2^24)."""
    rng = np.random.default_rng(6)
    counts, n, k = [3, 0, 9], 16, 24
    x, w, g, o = product_inputs(rng, counts, n, k, True)
    g = np.sign(g)
    d_o, y = [dev(o)], [torch.empty(12, n, dtype=torch.bfloat16, device="cuda")]
    dx, dw = [torch.empty(12, k, dtype=torch.bfloat16, device="cuda")], [torch.empty(3, n, k, device="cuda")]
    bf = torch.bfloat16
    lib.ccl_moe_product_grad_input([dev(g, bf)], d_o, [dev(w, bf)], dx)
    lib.ccl_moe_product_grad_weight([dev(g, bf)], [dev(x, bf)], d_o, dw)

    def total(xx, ww):
        lib.ccl_moe_product([dev(xx, bf)], d_o, [dev(ww, bf)], y)
        return (host(y[0]).astype(np.float64) * g).sum()

    # |y| <= 24 * 4 * 4 needs 9 bits: keep it below 256 so that bf16 holds it
    x, w = np.clip(x, -2, 2), np.clip(w, -2, 2)
    lib.ccl_moe_product_grad_input([dev(g, bf)], d_o, [dev(w, bf)], dx)
    lib.ccl_moe_product_grad_weight([dev(g, bf)], [dev(x, bf)], d_o, dw)
    for i, j in [(0, 0), (5, 23), (11, 7)]:
        up, down = x.copy(), x.copy()
        up[i, j] += 1
        down[i, j] -= 1
        assert (total(up, w) - total(down, w)) / 2 == host(dx[0])[i, j]
    for e, i, j in [(0, 0, 0), (2, 15, 23), (1, 3, 3)]:
        up, down = w.copy(), w.copy()
        up[e, i, j] += 1
        down[e, i, j] -= 1
        assert (total(x, up) - total(x, down)) / 2 == host(dw[0])[e, i, j]


def test_calls_on_another_stream_and_in_a_graph(lib):
    rng = np.random.default_rng(7)
    counts, n, k = [40, 100], 64, 128
    x, w, _, o = product_inputs(rng, counts, n, k, True)
    d_x, d_w, d_o = [dev(x, torch.bfloat16)], [dev(w, torch.bfloat16)], [dev(o)]
    y = [torch.zeros(140, n, dtype=torch.bfloat16, device="cuda")]
    rows = [torch.arange(140, dtype=torch.int32, device="cuda").flip(0).view(70, 2).contiguous()]
    out = [torch.zeros(70, n, dtype=torch.bfloat16, device="cuda")]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    lib.ccl_moe_product(d_x, d_o, d_w, y, stream=s)
    lib.ccl_moe_from_experts(y, rows, None, out, stream=s)
    s.synchronize()
    want = rounded(experts.product(x, o, w, np.zeros((140, n))), torch.bfloat16)
    assert torch.equal(y[0].cpu(), want)
    first = out[0].clone()
    y[0].zero_()
    out[0].zero_()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        lib.ccl_moe_product(d_x, d_o, d_w, y)
        lib.ccl_moe_from_experts(y, rows, None, out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[0].cpu(), want) and torch.equal(out[0], first)


def test_rows_past_32_bit_offsets(lib):
    """A buffer of more than 2^32 elements: the rows behind it are found."""
    hidden, tokens = 1 << 20, 2100
    x = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.arange(tokens, device="cuda") % 251
    x[:, -1] = torch.arange(tokens, device="cuda") % 241
    rows = [torch.stack([torch.arange(tokens), tokens + torch.arange(tokens).flip(0)], 1).to(torch.int32).cuda()]
    ordered = [torch.zeros(2 * tokens, hidden, dtype=torch.bfloat16, device="cuda")]
    lib.ccl_moe_to_experts([x], rows, ordered)
    assert torch.equal(ordered[0][:tokens], x) and torch.equal(ordered[0][tokens:], x.flip(0))
    out = [torch.empty_like(x)]
    lib.ccl_moe_from_experts(ordered, rows, None, out)
    assert torch.equal(out[0], x * 2)


def test_long_sums_keep_fp32_precision(lib):
    """An fp32 weight gradient over 20,000 rows.  The tensor core cuts its sums
    towards zero once per 16 rows, by half a unit in the last place (2^-24) on
    average; in parts of 512 rows that is at most 32 * 2^-24 of the result,
    where one sum would be off by 1250 * 2^-24.  Odd widths take the loaders."""
    rng = np.random.default_rng(10)
    for n, k in ((128, 256), (99, 131)):
        x, dy = bf16_exact(rng, (20000, k)), bf16_exact(rng, (20000, n))
        dw = [torch.empty(1, n, k, device="cuda")]
        lib.ccl_moe_product_grad_weight([dev(dy, torch.bfloat16)], [dev(x, torch.bfloat16)],
                                        [torch.tensor([0, 20000], dtype=torch.int32, device="cuda")], dw)
        want = dy.astype(np.float64).T @ x.astype(np.float64)
        assert np.linalg.norm(host(dw[0])[0] - want) <= 32 * 2.0 ** -24 * np.linalg.norm(want)


def test_refusals_of_the_binding(lib):
    """What the binding says of wrong tensors: lists, places, types, shapes, strides."""
    rows = [torch.zeros(4, 2, dtype=torch.int32, device="cuda")]
    y, out = [torch.zeros(8, 16, device="cuda")], [torch.zeros(4, 16, device="cuda")]
    w = [torch.ones(4, 2, device="cuda")]
    lib.ccl_moe_from_experts(y, rows, w, out)
    for args, said in [((y, [rows[0].long()], w, out), "int32"), ((y, [rows[0].cpu()], w, out), "CUDA"),
                       ((y * 2, rows, w, out), "1 rank buffers"), ((y, rows, w, [out[0][:3]]), "elements"),
                       ((y, rows, w, [out[0].bfloat16()]), "float32"), ((y, rows, [w[0].double()], out), "float32"),
                       (([torch.zeros(16, 8, device="cuda").T], rows, w, out), "contiguous"),
                       (([torch.zeros(8, 16, 1, device="cuda")], rows, w, out), "dimensions"),
                       (([3], rows, w, out), "must be a CUDA tensor"), (([], rows, w, out), "rank buffers"),
                       ((y, rows + [rows[0][:, :1].contiguous()], w, out), "dimensions"),
                       (([torch.zeros(8, 16, dtype=torch.float64, device="cuda")], rows, w, out), "float64")]:
        with pytest.raises(ValueError, match=said):
            lib.ccl_moe_from_experts(*args)
    with pytest.raises(lib.CclError, match="overlaps"):
        lib.ccl_moe_from_experts(y, rows, w, [y[0][:4]])
    with pytest.raises(lib.CclError, match="bf16"):
        lib.ccl_moe_to_experts([torch.zeros(4, 16, dtype=torch.int32, device="cuda")], rows,
                               [torch.zeros(8, 16, dtype=torch.int32, device="cuda")])
    with pytest.raises(ValueError, match="columns"):
        lib.ccl_moe_product([torch.zeros(4, 8, device="cuda").bfloat16()], rows, [torch.zeros(2, 8, 9, device="cuda").bfloat16()],
                            [torch.zeros(4, 8, device="cuda").bfloat16()])
    with pytest.raises(ValueError, match="must be a CUDA tensor$"):
        lib.ccl_moe_product([torch.zeros(4, 8).bfloat16().pin_memory()], rows, [torch.zeros(1, 8, 8, device="cuda").bfloat16()],
                            [torch.zeros(4, 8, device="cuda").bfloat16()])
    with pytest.raises(ValueError, match="dweights needs y"):
        lib.ccl_moe_from_experts_grad(out, None, rows, w, None, w)
