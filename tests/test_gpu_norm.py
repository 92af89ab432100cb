"""The layer norm and its gradients against the 64-bit definitions.

Tolerances count roundings of 2^-24.  A mean over n columns is off by at most
S = n / 32 + 32 of them (the additions in a row, and the joining) relative to the
mean magnitude; variance, and the two means of the gradient, likewise.  y's terms
are (v - mean) rstd w, whose factors carry S and a few more each, the mean's own
error times rstd w, and b; dx's are g, mean g and z mean(g z) times rstd, and dsum.
A weight's gradient is a sum over rows: one rounding per row that a thread adds and
per part that is joined, and those of z.  Each output is rounded once to its type.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import ccl
from oracle import router
from test_gpu_router import ONE, Buffer

pytestmark = pytest.mark.gpu
STEP = {"f32": ONE, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rounded(v: np.ndarray, dtype: str) -> np.ndarray:
    return torch.tensor(v).to(DT[dtype]).double().numpy()


SHAPES = [  # rows of each rank, columns
    ([1], 1), ([3], 2), ([5, 0, 2], 8), ([17], 31), ([9, 40], 64), ([33], 100), ([130], 128), ([7, 7], 257), ([64, 1, 5], 512), ([21], 1019),
    ([200, 77], 1024), ([30], 2047), ([40], 2048), ([11, 3], 2560), ([19], 4096), ([1], 5120), ([23], 7168), ([13], 7169), ([6], 8192),
    ([7], 12288), ([5], 12289), ([4, 2], 16383), ([9], 16384), ([700], 256),
]


@pytest.mark.parametrize("dtype,wt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,cols", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_norm(rows, cols, dtype, wt):
    c = ccl()
    rng = np.random.default_rng(cols)
    for off, residual, bias, stats in ((False, True, True, True), (True, False, True, False), (False, False, False, True), (True, True, False, True)):
        x = [rounded(rng.normal(size=(t, cols)) * 3 + 5, dtype) for t in rows]
        for v in x:
            if v.shape[0] > 2:
                v[1] = 7.0  # a constant row: nothing but the bias is left
        res = [rounded(rng.normal(size=v.shape), dtype) if residual else None for v in x]
        w, b = rounded(rng.normal(size=cols), wt), rounded(rng.normal(size=cols), wt)
        bx, br = [Buffer(v.shape, dtype, off, v) for v in x], [Buffer(v.shape, dtype, off, v) if residual else None for v in res]
        bw, bb = Buffer((cols,), wt, off, w), Buffer((cols,), wt, off, b)
        y, total = [Buffer(v.shape, dtype, off) for v in x], [Buffer(v.shape, dtype, off) for v in x]
        mean, rstd = [Buffer((t,), "f32") for t in rows], [Buffer((t,), "f32") for t in rows]
        c.ccl_layer_norm([q.t for q in bx], [bw.t] * len(rows), [bb.t] * len(rows) if bias else None, [q.t for q in y],
                         residual=[q.t for q in br] if residual else None, sum=[q.t for q in total] if residual else None,
                         mean=[q.t for q in mean] if stats else None, rstd=[q.t for q in rstd] if stats else None, eps=1e-3)
        S = (cols / 32 + 32) * ONE
        for r, v in enumerate(x):
            if not v.size:
                continue
            if residual:
                v = rounded((v + res[r]).astype(np.float32), dtype)  # fp32 sums of bf16 or fp32 values, rounded once
                np.testing.assert_array_equal(total[r].numpy(), v)
            want, m, s = router.norm(v, w, b if bias else None, 1e-3)
            level = np.abs(v).mean(1)
            # the mean's error enters every difference, and the variance by its square
            off_mean = S * level
            off_s = S + (off_mean * s) ** 2
            z = np.abs(v - m[:, None]) * s[:, None]
            bound = np.abs(w) * (z * (off_s + 4 * ONE)[:, None] + (off_mean * s)[:, None]) + 4 * ONE * (np.abs(b) if bias else 0.0)
            assert (np.abs(y[r].numpy() - want) <= bound + STEP[dtype] * np.abs(want)).all()
            if stats:
                assert (np.abs(mean[r].numpy() - m) <= off_mean).all()
                assert (np.abs(rstd[r].numpy() - s) <= (off_s + 4 * ONE) * s).all()


@pytest.mark.parametrize("dtype,wt,dw", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f32", "f32", "f32"), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("rows,cols", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_gradients(rows, cols, dtype, wt, dw):
    c = ccl()
    rng = np.random.default_rng(cols + 1)
    p = len(rows)
    for off, extra, weight, bias in ((False, True, True, True), (True, False, True, False), (False, False, False, True), (True, True, False, False),
                                     (False, False, True, True)):
        x = [rounded(rng.normal(size=(t, cols)) * 2 + 1, dtype) for t in rows]
        dy = [rounded(rng.normal(size=v.shape), dtype) for v in x]
        ds = [rounded(rng.normal(size=v.shape), dtype) for v in x]
        w = rounded(rng.normal(size=cols), wt)
        stats = [[s.astype(np.float32) for s in router.norm(v, w, None, 1e-3)[1:]] for v in x]
        bx, bd, bs = ([Buffer(v.shape, dtype, off, v) for v in vs] for vs in (x, dy, ds))
        mean, rstd = ([Buffer((t,), "f32", False, s[i]) for t, s in zip(rows, stats)] for i in (0, 1))
        bw = Buffer((cols,), wt, off, w)
        dx = [Buffer(v.shape, dtype, off) for v in x]
        gw, gb = [Buffer((cols,), dw, off) for _ in rows], [Buffer((cols,), dw, off) for _ in rows]
        c.ccl_layer_norm_grad([q.t for q in bd], [q.t for q in bx], [bw.t] * p, [q.t for q in mean], [q.t for q in rstd], [q.t for q in dx],
                              dsum=[q.t for q in bs] if extra else None, dweight=[q.t for q in gw] if weight else None,
                              dbias=[q.t for q in gb] if bias else None)
        S = (cols / 32 + 32) * ONE
        for r, v in enumerate(x):
            if v.size:
                m, s = stats[r]
                want, want_w, want_b = router.norm_grad(dy[r], v, w, m, s, ds[r] if extra else None)
                z, g, s = np.abs(v - m.astype(np.float64)[:, None]) * s[:, None], np.abs(dy[r] * w), s.astype(np.float64)[:, None]
                bound = s * (g + g.mean(1, keepdims=True) + z * (g * z).mean(1, keepdims=True)) * (S + 8 * ONE) + 2 * ONE * np.abs(ds[r] if extra else 0.0)
                # v - mean is rounded where they are close: against both
                near = ONE * (np.abs(v) + np.abs(m)[:, None]) * s
                bound = bound + s * near * (g * z).mean(1, keepdims=True) + s * z * (g * near).mean(1, keepdims=True)
                assert (np.abs(dx[r].numpy() - want) <= bound + STEP[dtype] * np.abs(want)).all()
                T = (v.shape[0] + 64) * ONE
                size_w = (np.abs(dy[r]) * z).sum(0) * (T + 8 * ONE) + (np.abs(dy[r]) * near).sum(0)
                size_b = np.abs(dy[r]).sum(0) * T
            else:
                want_w = want_b = np.zeros(cols)
                size_w = size_b = 0.0
            if weight:
                assert (np.abs(gw[r].numpy() - want_w) <= size_w + STEP[dw] * np.abs(want_w)).all()
            if bias:
                assert (np.abs(gb[r].numpy() - want_b) <= size_b + STEP[dw] * np.abs(want_b)).all()


def test_every_rank_has_its_own_weight():
    c = ccl()
    x = [torch.randn(6, 64, device="cuda") for _ in range(2)]
    w, b = [torch.randn(64, device="cuda") for _ in x], [torch.randn(64, device="cuda") for _ in x]
    y = [torch.empty_like(v) for v in x]
    c.ccl_layer_norm(x, w, b, y)
    for r, v in enumerate(x):
        z = (v.double() - v.double().mean(1, keepdim=True)) / (v.double().var(1, correction=0, keepdim=True) + 1e-5).sqrt()
        assert ((z * w[r].double() + b[r].double() - y[r]).abs() <= 64 * ONE * (z * w[r]).abs().clamp(min=1)).all()


def test_large_mean_keeps_the_variance():
    """The variance is taken around the mean, not as a difference of squares: rows
    of 4096 +- 1 in fp32, whose squares leave no bit for it."""
    c = ccl()
    x = torch.randn(8, 1024, device="cuda") + 4096
    y, mean, rstd = torch.empty_like(x), torch.empty(8, device="cuda"), torch.empty(8, device="cuda")
    one = torch.ones(1024, device="cuda")
    c.ccl_layer_norm([x], [one], None, [y], mean=[mean], rstd=[rstd])
    want = (x.double().var(1, correction=0) + 1e-5).rsqrt()
    # the mean is off by at most 64 roundings of 4096 (2^-6 of the deviation's 1), the variance by its square
    assert ((rstd - want).abs() <= 2.0 ** -12 * want * 1.5).all()


def test_not_a_number_stays_in_its_row():
    c = ccl()
    x = torch.randn(10, 96, device="cuda").bfloat16()
    x[3, 5], x[7] = float("nan"), float("inf")
    w = torch.ones(96, device="cuda")
    y, clean = torch.empty_like(x), torch.empty_like(x)
    c.ccl_layer_norm([x], [w], None, [y])
    c.ccl_layer_norm([x.nan_to_num(0, 0, 0)], [w], None, [clean])
    rest = [0, 1, 2, 4, 5, 6, 8, 9]
    assert torch.equal(y[rest], clean[rest]) and y[3].isnan().all() and y[7].isnan().all()


def test_same_bits_whatever_the_workspace_held_and_in_a_graph():
    c = ccl()
    torch.manual_seed(0)
    p, T, C = 3, 501, 640
    x = [torch.randn(T + r, C, device="cuda").bfloat16() for r in range(p)]
    dy = [torch.randn_like(v) for v in x]
    w = [torch.randn(C, device="cuda")] * p
    y, dx = [torch.empty_like(v) for v in x], [torch.empty_like(v) for v in x]
    mean, rstd = [torch.empty(T + r, device="cuda") for r in range(p)], [torch.empty(T + r, device="cuda") for r in range(p)]
    gw, gb = [torch.empty(C, device="cuda") for _ in range(p)], [torch.empty(C, device="cuda") for _ in range(p)]
    ws = torch.full((c.ccl_layer_norm_grad_workspace_bytes(p, C),), 0xFF, dtype=torch.uint8, device="cuda")

    def both(**kw):
        c.ccl_layer_norm(x, w, None, y, mean=mean, rstd=rstd)
        c.ccl_layer_norm_grad(dy, x, w, mean, rstd, dx, dweight=gw, dbias=gb, **kw)

    both(workspace=ws)
    outs = y + dx + mean + rstd + gw + gb
    first = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for t in outs:
        t.zero_()
    graph.replay()
    graph.replay()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for a, b in zip(first, outs):
        assert torch.equal(a, b)
    for t in outs:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    c.ccl_layer_norm(x, w, None, y, mean=mean, rstd=rstd, stream=side)
    c.ccl_layer_norm_grad(dy, x, w, mean, rstd, dx, dweight=gw, dbias=gb, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(first, outs):
        assert torch.equal(a, b)


def test_refusals():
    c = ccl()
    x, w = [torch.randn(4, 8, device="cuda")], [torch.ones(8, device="cuda")]
    y, s = [torch.empty_like(x[0])], [torch.empty(4, device="cuda")]
    with pytest.raises(c.CclError, match="residual and sum"):
        c.ccl_layer_norm(x, w, None, y, residual=[torch.randn(4, 8, device="cuda")])
    with pytest.raises(c.CclError, match="mean and rstd"):
        c.ccl_layer_norm(x, w, None, y, mean=s)
    with pytest.raises(c.CclError, match="overlaps"):
        c.ccl_layer_norm(x, w, None, x)
    with pytest.raises(c.CclError, match="eps"):
        c.ccl_layer_norm(x, w, None, y, eps=-1.0)
    with pytest.raises(ValueError, match="weight must hold 8"):
        c.ccl_layer_norm(x, [torch.ones(7, device="cuda")], None, y)
    with pytest.raises(ValueError, match="bias"):
        c.ccl_layer_norm(x, w, [torch.ones(8, device="cuda").bfloat16()], y)
    with pytest.raises(ValueError, match="contiguous"):
        c.ccl_layer_norm([torch.randn(8, 4, device="cuda").t()], w, None, y)
    big = [torch.empty(1, 16385, device="cuda")]
    with pytest.raises(c.CclError, match="16384"):
        c.ccl_layer_norm(big, [torch.ones(16385, device="cuda")], None, [torch.empty_like(big[0])])
    with pytest.raises(c.CclError, match="workspace"):
        c.ccl_layer_norm_grad(x, [torch.randn(4, 8, device="cuda")], w, s, [torch.ones(4, device="cuda")], y, dweight=[torch.empty(8, device="cuda")],
                              workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
