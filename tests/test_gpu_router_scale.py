"""The norm and the router on many rows, many ranks and past 32-bit offsets, against
the definitions in 64 bits on the GPU; tolerances as in test_gpu_norm and
test_gpu_router."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from gpu_util import ccl
from test_gpu_router import ONE

pytestmark = pytest.mark.gpu
HALF = {torch.float32: ONE, torch.bfloat16: 2.0 ** -8}


def norm64(x, w, b, eps):
    v = x.double()
    mean = v.mean(1, keepdim=True)
    rstd = ((v - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    return (v - mean) * rstd * w.double() + (0.0 if b is None else b.double()), mean, rstd


def check_norm(y, x, w, b, eps):
    want, mean, rstd = norm64(x, w, b, eps)
    S = (x.shape[1] / 32 + 32) * ONE
    off_mean = S * x.double().abs().mean(1, keepdim=True) * rstd
    z = (x.double() - mean).abs() * rstd
    bound = w.double().abs() * (z * (S + off_mean.square() + 4 * ONE) + off_mean) + (0.0 if b is None else 4 * ONE * b.double().abs())
    assert ((y.double() - want).abs() <= bound + HALF[y.dtype] * want.abs()).all()


def check_norm_grad(dx, dy, x, w, mean, rstd, ds):
    v, d, m, s = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    z, g = (v - m) * s, d * w.double()
    want = s * (g - g.mean(1, keepdim=True) - z * (g * z).mean(1, keepdim=True)) + (0.0 if ds is None else ds.double())
    a, S = g.abs(), (x.shape[1] / 32 + 40) * ONE
    near = ONE * (v.abs() + m.abs()) * s
    bound = s * ((a + a.mean(1, keepdim=True) + z.abs() * (a * z.abs()).mean(1, keepdim=True)) * S + near * (a * z.abs()).mean(1, keepdim=True)
                 + z.abs() * (a * near).mean(1, keepdim=True)) + (0.0 if ds is None else 2 * ONE * ds.double().abs())
    assert ((dx.double() - want).abs() <= bound + HALF[dx.dtype] * want.abs()).all()
    return z, near


@pytest.mark.parametrize("rows,cols,dt", [(60001, 256, torch.bfloat16), (30011, 1024, torch.bfloat16), (9001, 5888, torch.bfloat16),
                                          (9001, 6144, torch.bfloat16), (9001, 7168, torch.bfloat16), (8003, 6144, torch.float32),
                                          (4001, 16384, torch.bfloat16), (20011, 1019, torch.bfloat16), (20011, 1019, torch.float32)])
def test_many_rows(rows, cols, dt):
    """Rows enough for the weights to be staged, with and without a bias."""
    c = ccl()
    torch.manual_seed(cols)
    x, dy, ds = ((torch.randn(rows, cols, device="cuda") + a).to(dt) for a in (0.5, 0.0, 0.0))
    w, b = torch.randn(cols, device="cuda").to(dt), torch.randn(cols, device="cuda").to(dt)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    for bias in (b, None):
        c.ccl_layer_norm([x], [w], None if bias is None else [bias], [y], mean=[mean], rstd=[rstd])
        check_norm(y, x, w, bias, 1e-5)
    gw, gb = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    for extra in (ds, None):
        c.ccl_layer_norm_grad([dy], [x], [w], [mean], [rstd], [y], dsum=None if extra is None else [extra], dweight=[gw], dbias=[gb])
        z, near = check_norm_grad(y, dy, x, w, mean, rstd, extra)
    d, T = dy.double(), (rows + 64) * ONE
    assert ((gw.double() - (d * z).sum(0)).abs() <= (d * z).abs().sum(0) * (T + 8 * ONE) + (d.abs() * near).sum(0) + ONE * gw.double().abs()).all()
    assert ((gb.double() - d.sum(0)).abs() <= d.abs().sum(0) * T).all()


@pytest.mark.parametrize("with_sum", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(2003, 8193), (2003, 8200), (2003, 12288), (2003, 16383), (2003, 16384), (9001, 61), (9001, 129), (9001, 513), (9001, 1025),
                                       (4001, 2049), (4001, 4097), (4001, 4104), (4001, 5120), (4001, 5128), (4001, 7168), (4001, 8192)])
def test_sums_over_many_rows(rows, cols, dt, with_sum):
    """The gradients of rows whose sums are kept in shared memory, and of every width of
    rows off the grid; two of each call give the same bits."""
    c = ccl()
    torch.manual_seed(cols)
    x, dy, ds = (torch.randn(rows, cols, device="cuda").to(dt) for _ in range(3))
    w = torch.randn(cols, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    c.ccl_layer_norm([x], [w], None, [y], mean=[mean], rstd=[rstd])
    check_norm(y, x, w, None, 1e-5)
    extra, got = ds if with_sum else None, []
    for _ in range(2):
        out = [torch.full_like(x, 3.0), torch.full((cols,), 3.0, device="cuda"), torch.full((cols,), 3.0, device="cuda")]
        c.ccl_layer_norm_grad([dy], [x], [w], [mean], [rstd], out[:1], dsum=None if extra is None else [extra], dweight=out[1:2], dbias=out[2:])
        got.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    dx, gw, gb = got[0]
    z, near = check_norm_grad(dx, dy, x, w, mean, rstd, extra)
    d, T = dy.double(), (rows + 64) * ONE
    assert ((gw.double() - (d * z).sum(0)).abs() <= (d * z).abs().sum(0) * (T + 8 * ONE) + (d.abs() * near).sum(0) + ONE * gw.double().abs()).all()
    assert ((gb.double() - d.sum(0)).abs() <= d.abs().sum(0) * T).all()


@pytest.mark.parametrize("dt,wt", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("rows,cols", [(5, 256), (20_011, 512), (3, 7168), (9001, 4096)])
def test_weights_off_the_grid_of_rows_on_it(rows, cols, dt, wt):
    """Weight and bias one element off 16 bytes, as a view into a flat buffer may be,
    few rows and many."""
    c = ccl()
    torch.manual_seed(cols)
    x, dy = torch.randn(rows, cols, device="cuda").to(dt), torch.randn(rows, cols, device="cuda").to(dt)
    w, b = (torch.randn(cols + 1, device="cuda").to(wt)[1:] for _ in range(2))
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    c.ccl_layer_norm([x], [w], [b], [y], mean=[mean], rstd=[rstd])
    check_norm(y, x, w, b, 1e-5)
    c.ccl_layer_norm_grad([dy], [x], [w], [mean], [rstd], [y])
    check_norm_grad(y, dy, x, w, mean, rstd, None)


def test_a_workspace_that_is_not_needed_is_left_alone():
    """The C call without dweight and dbias takes any workspace, and writes none."""
    import ctypes

    c = ccl()
    x, w = torch.randn(40, 64, device="cuda"), torch.ones(64, device="cuda")
    mean, rstd, dx = torch.zeros(40, device="cuda"), torch.ones(40, device="cuda"), torch.empty(40, 64, device="cuda")
    held = torch.full((1 << 20,), 5.0, device="cuda")
    one = lambda t: (ctypes.c_void_p * 1)(t.data_ptr())  # noqa: E731
    got = c.LIB.ccl_layer_norm_grad(one(x), None, one(x), one(w), one(mean), one(rstd), (ctypes.c_size_t * 1)(40), 1, 64, 0, 0, one(dx), 0, None, None,
                                    held[1024:].data_ptr(), 16, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert got == c.CCL_OK and (held == 5.0).all()


def test_sixty_four_ranks():
    c = ccl()
    torch.manual_seed(0)
    p, C, E, k = 64, 200, 24, 3
    rows = [(r * 7) % 13 for r in range(p)]  # some have none
    x = [torch.randn(t, C, device="cuda") for t in rows]
    w, b = [torch.randn(C, device="cuda") for _ in x], [torch.randn(C, device="cuda") for _ in x]
    res, y, total = [torch.randn_like(v) for v in x], [torch.empty_like(v) for v in x], [torch.empty_like(v) for v in x]
    mean, rstd = [torch.empty(t, device="cuda") for t in rows], [torch.empty(t, device="cuda") for t in rows]
    c.ccl_layer_norm(x, w, b, y, residual=res, sum=total, mean=mean, rstd=rstd)
    dx, gw, gb = [torch.empty_like(v) for v in x], [torch.full_like(v, 9.0) for v in w], [torch.full_like(v, 9.0) for v in w]
    c.ccl_layer_norm_grad(res, total, w, mean, rstd, dx, dsum=x, dweight=gw, dbias=gb)
    logits = [torch.randn(t, E, device="cuda") for t in rows]
    ids, gates = [torch.empty(t, k, dtype=torch.int32, device="cuda") for t in rows], [torch.empty(t, k, device="cuda") for t in rows]
    counts, losses, dl = [torch.empty(E + 1, dtype=torch.int32, device="cuda") for _ in rows], [torch.empty(1, device="cuda") for _ in rows], \
        [torch.empty_like(v) for v in logits]
    c.ccl_moe_gate(logits, ids, gates, counts=counts, losses=losses)
    c.ccl_moe_gate_grad(logits, ids, gates, dl, counts=counts, dlosses=losses)
    for r, t in enumerate(rows):
        if t == 0:
            assert (gw[r] == 0).all() and (gb[r] == 0).all() and (counts[r] == 0).all() and losses[r] == 0
            continue
        assert torch.equal(total[r], x[r] + res[r])
        check_norm(y[r], total[r], w[r], b[r], 1e-5)
        check_norm_grad(dx[r], res[r], total[r], w[r], mean[r], rstd[r], x[r])
        assert ((gb[r].double() - res[r].double().sum(0)).abs() <= 80 * ONE * res[r].double().abs().sum(0)).all()
        top = logits[r].sort(dim=1, descending=True, stable=True)
        assert torch.equal(ids[r].long(), top.indices[:, :k])
        assert int(counts[r][-1]) == t and int(counts[r][:-1].sum()) == t * k
        # one rank at a time gives the same
        one = torch.empty_like(dl[r])
        c.ccl_moe_gate_grad([logits[r]], [ids[r]], [gates[r]], [one], counts=[counts[r]], dlosses=[losses[r]])
        assert torch.equal(one, dl[r])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,experts,k", [(131077, 256, 8), (70001, 60, 6), (40003, 61, 8), (100003, 8, 2), (20001, 384, 8), (30001, 160, 12)])
def test_many_tokens(tokens, experts, k, dt):
    c = ccl()
    torch.manual_seed(experts)
    l = (torch.randn(tokens, experts, device="cuda") * 2).to(dt)
    l[::3] = (l[::3] * 2).round() / 2  # many equal ones
    l[5::17, experts // 3] = -math.inf
    l[-1000:] = -math.inf
    ids, gates = torch.empty(tokens, k, dtype=torch.int32, device="cuda"), torch.empty(tokens, k, device="cuda")
    counts, loss = torch.empty(experts + 1, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
    c.ccl_moe_gate([l], [ids], [gates], counts=[counts], losses=[loss])
    top, at = (l.double() + 0.0).sort(dim=1, descending=True, stable=True)
    want = torch.where(top[:, :k] == -math.inf, -1, at[:, :k]).int()
    assert torch.equal(ids, want)
    u = torch.exp(top[:, :k] - top[:, :1].clamp(min=-1e30)).nan_to_num(0.0)
    g = u / u.sum(1, keepdim=True).clamp(min=1e-300)
    A = (top[:-1000, :1] - top[:-1000].clamp(min=-60)).amax()
    tol = float((4 * A + experts / 8 + 32) * ONE)
    assert ((gates.double() - g).abs() <= tol * g + 1e-38).all()
    live = tokens - 1000
    n = torch.bincount(want[want >= 0].long(), minlength=experts)
    assert torch.equal(counts[:-1].long(), n) and int(counts[-1]) == live
    share = torch.softmax(l[:live].double(), 1)
    target = float((n * share.sum(0)).sum() * experts / (k * live * live))
    assert abs(float(loss) - target) <= (tol + (tokens / 1000 + 200) * ONE) * target  # a warp adds up to so many rows
    d = torch.randn(tokens, k, device="cuda")
    out = torch.empty_like(l)
    c.ccl_moe_gate_grad([l], [ids], [d], [out], counts=[counts])
    d = torch.where(want < 0, 0.0, d).double()
    own = g * (d - (g * d).sum(1, keepdim=True))
    a = n.double() * experts / (k * live * live)
    a = a - a.mean()
    full = torch.zeros(tokens, experts + 1, dtype=torch.float64, device="cuda").scatter_add_(1, torch.where(want < 0, experts, want).long(), own)[:, :-1]
    full[:live] += share * (a - (share * a).sum(1, keepdim=True))
    size = torch.zeros(tokens, experts + 1, dtype=torch.float64, device="cuda").scatter_add_(
        1, torch.where(want < 0, experts, want).long(), g * (d.abs() + (g * d.abs()).sum(1, keepdim=True)))[:, :-1]
    size[:live] += share * (a.abs() + (share * a.abs()).sum(1, keepdim=True))
    assert ((out.double() - full).abs() <= 2 * tol * size + HALF[dt] * full.abs() + 1e-38).all()


def test_rows_past_32_bit_offsets():
    """4.32e9 bf16 elements: element and byte offsets pass 2^32."""
    c = ccl()
    rows, cols = 600_011, 7200
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    y = torch.empty_like(x)
    w = torch.randn(cols, device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    c.ccl_layer_norm([x], [w], None, [y], mean=[mean], rstd=[rstd])
    for part in (slice(0, 300), slice(298_200, 298_500), slice(rows - 300, rows)):
        check_norm(y[part], x[part], w, None, 1e-5)
    gb = torch.empty(cols, device="cuda")
    c.ccl_layer_norm_grad([x], [x], [w], [mean], [rstd], [y], dbias=[gb])
    for part in (slice(0, 300), slice(298_200, 298_500), slice(rows - 300, rows)):
        check_norm_grad(y[part], x[part], x[part], w, mean[part], rstd[part], None)
    total = torch.zeros(cols, dtype=torch.float64, device="cuda")
    for at in range(0, rows, 50_000):
        total += x[at:at + 50_000].double().sum(0)
    # parts of some 4000 rows, by 0.8 on average
    assert ((gb.double() - total).abs() <= (rows / 152 + 400) * ONE * 0.9 * rows).all()


def test_logits_past_32_bit_offsets():
    c = ccl()
    tokens, experts, k = 16_900_003, 256, 2
    l = torch.empty(tokens, experts, dtype=torch.bfloat16, device="cuda").normal_()
    ids, gates = torch.empty(tokens, k, dtype=torch.int32, device="cuda"), torch.empty(tokens, k, device="cuda")
    counts, loss = torch.empty(experts + 1, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
    c.ccl_moe_gate([l], [ids], [gates], counts=[counts], losses=[loss])
    out = torch.empty_like(l)
    c.ccl_moe_gate_grad([l], [ids], [gates], [out])
    for part in (slice(0, 2000), slice(8_388_000, 8_390_000), slice(16_776_000, 16_778_000), slice(tokens - 2000, tokens)):
        top, at = l[part].double().sort(dim=1, descending=True, stable=True)
        assert torch.equal(ids[part].long(), at[:, :k])
        g = torch.softmax(top[:, :k], 1)
        assert ((gates[part].double() - g).abs() <= 128 * ONE * g).all()
        d = gates[part].double()
        want = torch.zeros(2000, experts, dtype=torch.float64, device="cuda").scatter_(1, at[:, :k], g * (d - (g * d).sum(1, keepdim=True)))
        assert ((out[part].double() - want).abs() <= 256 * ONE + 2.0 ** -8 * want.abs()).all()
    assert int(counts[-1]) == tokens and int(counts[:-1].long().sum()) == tokens * k and abs(float(loss) - 1.0) < 0.01


def test_nothing_but_empty_ranks():
    c = ccl()
    l, ids = [torch.empty(0, 8, device="cuda")] * 2, [torch.empty(0, 2, dtype=torch.int32, device="cuda")] * 2
    gates = [torch.empty(0, 2, device="cuda")] * 2
    for call in (lambda n, v: c.ccl_moe_gate(l, ids, gates, counts=n, losses=v), lambda n, v: c.ccl_moe_balance(l, ids, n, v, together=True)):
        n, v = [torch.full((9,), 7, dtype=torch.int32, device="cuda") for _ in l], [torch.full((1,), 7.0, device="cuda") for _ in l]
        call(n, v)
        assert all((a == 0).all() for a in n) and all((a == 0).all() for a in v)
    c.ccl_moe_gate(l, ids, gates)
    c.ccl_moe_gate_grad(l, ids, gates, [torch.empty(0, 8, device="cuda")] * 2)
    c.ccl_moe_balance_grad(l, n, [torch.empty(0, 8, device="cuda")] * 2, 2)
    x, w = [torch.empty(0, 16, device="cuda")], [torch.ones(16, device="cuda")]
    none = [torch.empty(0, device="cuda")]
    c.ccl_layer_norm(x, w, None, [torch.empty(0, 16, device="cuda")])
    g = [torch.full((16,), 7.0, device="cuda")]
    c.ccl_layer_norm_grad(x, x, w, none, none, [torch.empty(0, 16, device="cuda")], dweight=g)
    assert (g[0] == 0).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_nan_of_either_sign_comes_first(dt):
    c = ccl()
    l = torch.randn(40, 64, device="cuda").to(dt)
    bits = l.view(torch.int16 if dt == torch.bfloat16 else torch.int32)
    bits[3, 9] = -64 if dt == torch.bfloat16 else -4194304  # 0xFFC0...
    bits[4, 9] = 0x7FFF if dt == torch.bfloat16 else 0x7FFFFFFF
    bits[5, 9], bits[5, 4] = -1, -1  # all ones, twice
    ids, gates = torch.empty(40, 3, dtype=torch.int32, device="cuda"), torch.empty(40, 3, device="cuda")
    c.ccl_moe_gate([l], [ids], [gates])
    assert ids[3, 0] == 9 and ids[4, 0] == 9 and ids[5, 0] == 4 and ids[5, 1] == 9
    assert gates[3:6].isnan().all() and not gates[:3].isnan().any() and not gates[6:].isnan().any()


def test_workspace_of_another_stream_s_call():
    """A call on a stream that is not the current one brings its own workspace from there."""
    c = ccl()
    torch.manual_seed(3)
    side = torch.cuda.Stream()
    l = [torch.randn(5000, 64, device="cuda")]
    ids, gates = [torch.empty(5000, 4, dtype=torch.int32, device="cuda")], [torch.empty(5000, 4, device="cuda")]
    counts, losses = [torch.empty(65, dtype=torch.int32, device="cuda")], [torch.empty(1, device="cuda")]
    c.ccl_moe_gate(l, ids, gates, counts=counts, losses=losses)
    want = [counts[0].clone(), losses[0].clone()]
    torch.cuda.synchronize()
    held = torch.cuda.memory_stats()["active.all.current"]
    for handle in (side, torch.cuda.ExternalStream(side.cuda_stream)):
        for _ in range(20):
            c.ccl_moe_gate(l, ids, gates, counts=counts, losses=losses, stream=handle)
    torch.cuda.synchronize()
    assert torch.equal(counts[0], want[0]) and torch.equal(losses[0], want[1])
    assert torch.cuda.memory_stats()["active.all.current"] == held
