"""Pins of the experts' and the optimizer's oracles, independent of their code."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import adamw, experts


def test_sort_by_hand():
    # tokens 0..2 with two choices; experts 4..6 belong to the rank
    ids = np.array([[5, 4], [9, 5], [6, 5]])
    offsets, rows = experts.sort(ids, 3, first=4)
    assert offsets.tolist() == [0, 1, 4, 5]
    assert rows.tolist() == [[1, 0], [-1, 2], [4, 3]]


@pytest.mark.parametrize("tokens,k,num", [(1, 1, 1), (40, 3, 7), (200, 8, 64)])
def test_sort_is_numpys_stable_sort(tokens, k, num):
    ids = np.random.default_rng(tokens).integers(0, num, (tokens, k))
    offsets, rows = experts.sort(ids, num)
    order = np.argsort(ids.reshape(-1), kind="stable")
    assert (rows.reshape(-1)[order] == np.arange(ids.size)).all()
    assert (np.diff(offsets) == np.bincount(ids.reshape(-1), minlength=num)).all()


def test_rows_and_products_against_autograd():
    rng = np.random.default_rng(0)
    tokens, k, num, h, n = 11, 3, 5, 6, 4
    ids = rng.integers(0, num, (tokens, k))
    offsets, rows = experts.sort(ids, num)
    x = torch.tensor(rng.standard_normal((tokens, h)), requires_grad=True)
    w = torch.tensor(rng.standard_normal((num, n, h)), requires_grad=True)
    gates = torch.tensor(rng.random((tokens, k)), requires_grad=True)
    ordered = x[torch.tensor(np.argsort(ids.reshape(-1), kind="stable") // k)]
    y = torch.cat([ordered[offsets[e]:offsets[e + 1]] @ w[e].T for e in range(num)])
    y.retain_grad()
    ordered.retain_grad()
    out = (y[torch.tensor(rows)] * gates[..., None]).sum(1)
    dout = rng.standard_normal(out.shape)
    out.backward(torch.tensor(dout))
    g = dict(rtol=1e-12, atol=1e-12)
    mine = experts.to_experts(x.detach().numpy(), rows, np.zeros((tokens * k, h)))
    np.testing.assert_array_equal(mine, ordered.detach().numpy())
    my = experts.product(mine, offsets, w.detach().numpy(), np.zeros((tokens * k, n)))
    np.testing.assert_allclose(my, y.detach().numpy(), **g)
    np.testing.assert_allclose(experts.from_experts(my, rows, gates.detach().numpy())[0], out.detach().numpy(), **g)
    dy, dw, _ = experts.from_experts_grad(dout, my, rows, gates.detach().numpy(), np.zeros_like(my))
    np.testing.assert_allclose(dy, y.grad.numpy(), **g)
    np.testing.assert_allclose(dw, gates.grad.numpy(), **g)
    dx = experts.product_grad_input(dy, offsets, w.detach().numpy(), np.zeros_like(mine))
    np.testing.assert_allclose(dx, ordered.grad.numpy(), **g)
    np.testing.assert_allclose(experts.product_grad_weight(dy, mine, offsets), w.grad.numpy(), **g)
    np.testing.assert_allclose(experts.from_experts(dx, rows, None)[0], x.grad.numpy(), **g)


def test_adamw_formula_against_torch():
    rng = np.random.default_rng(1)
    h = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    p = torch.tensor(rng.standard_normal(50), requires_grad=True)
    opt = torch.optim.AdamW([p], **h)
    mine, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for step in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.tensor(g)
        opt.step()
        mine, m, v = adamw.step64(mine, g, m, v, step, **h)
        np.testing.assert_allclose(mine, p.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_step32_follows_step64():
    # m and v: 3 roundings each; the update 8 more; far below 2^-19 of the largest term
    rng = np.random.default_rng(2)
    p, g, m = (rng.standard_normal(1000).astype(np.float32) for _ in range(3))
    v = rng.random(1000).astype(np.float32)
    h = dict(step=7, lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01)
    a, b = adamw.step32(p, g, m, v, **h), adamw.step64(p, g, m, v, **h)
    for x, y in zip(a[:2], b[:2]):
        assert np.abs(x - y).max() <= 2.0 ** -19 * 5
    assert (np.abs(a[2] - b[2]) <= 2.0 ** -22 * b[2]).all()


def test_codes_of_m_are_torchs_e4m3_of_the_scaled_block():
    x = np.random.default_rng(3).standard_normal(1000).astype(np.float32)
    codes, scales = adamw.encode_m(x)
    for b in range(8):
        part = x[128 * b:128 * b + 128]
        top = np.abs(part).max()
        want = torch.from_numpy(part * (np.float32(448) * (np.float32(1) / top))).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert (codes[128 * b:128 * b + 128] == want.view(torch.uint8).numpy()).all()
        assert scales[b] == top * (np.float32(1) / np.float32(448))


def test_thresholds_average_out_over_steps():
    """Over 1000 steps an element's thresholds are spread evenly (golden-ratio
    sequence: the discrepancy of 1000 points is below 1 %), so a value held
    still is coded right on average, where nearest rounding would be off by up
    to half a spacing."""
    u = np.stack([adamw.thresholds(64, s) for s in range(1, 1001)]) / 2.0 ** 20
    for q in (0.1, 0.25, 0.5, 0.9):
        assert np.abs((u < q).mean(0) - q).max() < 0.01
    root = np.full(128, 0.61, dtype=np.float32)
    root[0] = 1.0  # the block's amax
    mean = np.mean([adamw.decode(*adamw.encode_root(root, root ** 2, s)) for s in range(1, 1001)], axis=0)
    # spacing at 0.61 is 2^-4 of the amax's power of two: 448 * 0.61 = 273 lies in [256, 448], spacing 32 / 448
    assert np.abs(mean - root)[1:].max() < 0.01 * 32 / 448


def test_codes_of_root_neighbour_the_value_and_spare_zero_for_zero():
    rng = np.random.default_rng(4)
    root = np.exp(rng.standard_normal(3000) * 6).astype(np.float32)
    root[5:9] = 0
    codes, scales = adamw.encode_root(root, root, 12)
    got = adamw.decode(codes, scales)
    assert (codes[5:9] == 0).all() and (np.delete(codes, range(5, 9)) > 0).all()
    s = np.repeat(scales, 128)[:3000]
    # within one spacing (2^-3 relative, 2^-9 scales at the bottom), the scale's own rounding aside
    assert (np.abs(got - root) <= np.maximum(root * 2.0 ** -3, s * 2.0 ** -9) * (1 + 1e-5)).all()


def test_values_that_are_not_finite_stay_with_their_element():
    x = np.ones(256, dtype=np.float32)
    x[3], x[7], x[200] = np.inf, np.nan, -np.inf
    for codes, scales in (adamw.encode_m(x), adamw.encode_root(np.abs(x), np.abs(x), 3)):
        assert (codes[[3, 7, 200]] == 0x7F).all()
        fine = np.delete(np.arange(256), [3, 7, 200])
        np.testing.assert_allclose(adamw.decode(codes, scales)[fine], 1.0, rtol=1e-6)
