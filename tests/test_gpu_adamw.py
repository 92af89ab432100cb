"""GPU parity of the AdamW step: bit for bit with the fp32 oracle, close to the 64-bit one.

Against 64 bits, in units of fp32's rounding 2^-24, a factor that is itself
rounded to fp32 counting a half: m takes 2.5 of |b1 m| + |(1 - b1) g| and v 3.5
of itself, both below 2^-22; the parameter 1.5 of its old value and 1 for the
last sum, below 2^-22; the update 10.3 (m 2.5, the root 2.75, its factor 1.5,
eps 1, the quotient 1, the step size 1.5) and 1 for the last sum, below 2^-20;
a bf16 parameter 2^-8, its rounding unit, of the result more.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import ccl
from oracle import adamw

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
H = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def optim():
    ccl()
    from a2a_ring_ordered_gb300 import optim as mod

    return mod


def held(a, dtype):
    """a's values as dtype holds them, fp32."""
    return torch.from_numpy(a).to(DT[dtype]).float().numpy()


def place(a, dtype, off):
    store = torch.zeros(a.size + off + 16, dtype=dtype, device="cuda")
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    store[off:off + a.size] = t.view(dtype) if dtype == torch.float8_e4m3fn else t.to(dtype)
    return store[off:off + a.size]


def zeroed_ends(t, off):
    s = t._base.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t._base
    return bool((s[:off] == 0).all() and (s[off + t.numel():] == 0).all())


SIZES = [[1], [127, 128, 129], [4096, 4097, 1, 0, 5000], [3, 300, 30001], [17] * 60]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,copy", [("f32", "bf16", True), ("f32", "f32", False), ("bf16", "bf16", False),
                                             ("bf16", "f32", False)])
@pytest.mark.parametrize("off", [0, 1, 3, 4])
@pytest.mark.parametrize("sizes", SIZES)
def test_step(optim, sizes, off, param, grad, copy, bits):
    rng = np.random.default_rng(len(sizes) + off)
    P = [held(rng.standard_normal(n).astype(np.float32), param) for n in sizes]
    G = [held((rng.standard_normal(n) * np.exp(rng.standard_normal(n))).astype(np.float32), grad) for n in sizes]
    M = [(rng.standard_normal(n)).astype(np.float32) for n in sizes]
    V = [(rng.standard_normal(n) ** 2).astype(np.float32) for n in sizes]
    step = 4
    if bits == 8:
        mc = [adamw.encode_m(m) for m in M]
        vc = [adamw.encode_root(np.sqrt(v), v, step) for v in V]
        M = [adamw.decode(*c) for c in mc]
        V = [adamw.decode(*c) for c in vc]
        V = [v * v for v in V]
        states = {"exp_avg": [place(c, torch.float8_e4m3fn, off) for c, _ in mc],
                  "exp_avg_sq": [place(c, torch.float8_e4m3fn, off) for c, _ in vc],
                  "exp_avg_scale": [place(s, torch.float32, 1) for _, s in mc],
                  "exp_avg_sq_scale": [place(s, torch.float32, 1) for _, s in vc]}
    else:
        states = {"exp_avg": [place(m, torch.float32, off) for m in M],
                  "exp_avg_sq": [place(v, torch.float32, off) for v in V]}
    params = [place(p, DT[param], off) for p in P]
    copies = [place(np.zeros(n, np.float32), torch.bfloat16, off) for n in sizes] if copy else None
    opt = optim.AdamW(params, [place(g, DT[grad], off) for g in G], **H, state_bits=bits, states=states, copies=copies, step=step)
    opt.step()
    torch.cuda.synchronize()
    for i, n in enumerate(sizes):
        p, m, v, root = adamw.step32(P[i], G[i], M[i], V[i], step + 1, **H)
        got = params[i].float().cpu().numpy()
        np.testing.assert_array_equal(got, held(p, param))
        if copy:
            np.testing.assert_array_equal(copies[i].float().cpu().numpy(), held(p, "bf16"))
        if bits == 32:
            np.testing.assert_array_equal(states["exp_avg"][i].cpu().numpy(), m)
            np.testing.assert_array_equal(states["exp_avg_sq"][i].cpu().numpy(), v)
        else:
            for name, want in (("exp_avg", adamw.encode_m(m)), ("exp_avg_sq", adamw.encode_root(root, v, step + 1))):
                np.testing.assert_array_equal(states[name][i].view(torch.uint8).cpu().numpy(), want[0])
                np.testing.assert_array_equal(states[name + "_scale"][i].cpu().numpy(), want[1])
        # the formula in 64 bits
        p64, m64, v64 = adamw.step64(P[i], G[i], M[i], V[i], step + 1, **H)
        b1, b2 = H["betas"]
        assert (np.abs(m - m64) <= 2.0 ** -22 * (np.abs(b1 * M[i]) + np.abs((1 - b1) * G[i]))).all()
        assert (np.abs(v - v64) <= 2.0 ** -22 * v64).all()
        update = H["lr"] * (np.abs(b1 * M[i]) + np.abs((1 - b1) * G[i])) / (1 - b1 ** (step + 1)) / (np.sqrt(v64 / (1 - b2 ** (step + 1))) + H["eps"])
        half = 2.0 ** -8 * 1.001 if param == "bf16" else 0.0
        assert (np.abs(got - p64) <= 2.0 ** -22 * np.abs(P[i]) + 2.0 ** -20 * update + half * (np.abs(P[i]) + update)).all()
        for name, ts in {"param": params, "copy": copies or params, **states}.items():
            assert zeroed_ends(ts[i], 1 if name.endswith("scale") else off)


def test_many_tensors_take_more_than_one_launch(optim):
    lib = ccl()
    rng = np.random.default_rng(0)
    P = [rng.standard_normal(1 + i % 5).astype(np.float32) for i in range(1000)]
    params = [torch.from_numpy(p).cuda() for p in P]
    grads = [torch.ones_like(p) for p in params]
    opt = optim.AdamW(params, grads, **H)
    before = lib.ccl_kernel_launch_count()
    opt.step()
    assert lib.ccl_kernel_launch_count() - before == 3
    for p, old in zip(params, P):
        z = np.zeros_like(old)
        np.testing.assert_array_equal(p.cpu().numpy(), adamw.step32(old, z + 1, z, z, 1, **H)[0])


def test_grad_scale_and_learning_rate_of_a_step(optim):
    rng = np.random.default_rng(1)
    p0, g0 = rng.standard_normal(1000).astype(np.float32), rng.standard_normal(1000).astype(np.float32)
    p, z = torch.from_numpy(p0).cuda(), np.zeros(1000, np.float32)
    opt = optim.AdamW([p], [torch.from_numpy(g0).cuda()], **H)
    opt.step(lr=0.5, grad_scale=torch.tensor([0.3], device="cuda"))
    want = adamw.step32(p0, g0, z, z, 1, **{**H, "lr": 0.5}, grad_scale=np.float32(0.3))
    np.testing.assert_array_equal(p.cpu().numpy(), want[0])
    np.testing.assert_array_equal(opt.moments(0)[1].cpu().numpy(), want[2])


@pytest.mark.parametrize("bits", [32, 8])
def test_values_that_are_not_finite_stay_in_their_element(optim, bits):
    g = torch.full((300,), 0.5, device="cuda")
    g[5], g[130], g[299] = float("nan"), float("inf"), 1e30
    p = torch.ones(300, device="cuda")
    opt = optim.AdamW([p], [g], **H, state_bits=bits)
    for _ in range(3):
        opt.step()
    bad = {5, 130, 299}
    fine = [i for i in range(300) if i not in bad]
    assert torch.isfinite(p[fine]).all() and torch.isnan(p[5])
    m, v = opt.moments(0)
    assert torch.isfinite(m[fine]).all() and torch.isfinite(v[fine]).all()
    assert (p[fine] < 1).all()


def test_zero_gradients_leave_zero_states(optim):
    p = torch.ones(200, device="cuda")
    opt = optim.AdamW([p], [torch.zeros(200, device="cuda")], **H, state_bits=8)
    opt.step()
    assert all((t.view(torch.uint8) == 0).all() for n in ("exp_avg", "exp_avg_sq") for t in opt.table.tensors[n])
    assert all((t == 1).all() for n in ("exp_avg_scale", "exp_avg_sq_scale") for t in opt.table.tensors[n])
    np.testing.assert_array_equal(p.cpu().numpy(), np.full(200, np.float32(1) * np.float32(1 - 1e-2 * 0.1)))


def test_8_bit_states_train_as_32_bit_ones_do(optim):
    """Least squares with noisy gradients whose size changes by 100 midway: v has
    to follow it up and down, which codes rounded to nearest would not (a step
    of beta2 = 0.999 moves sqrt(v) by at most 0.05 %, a code's spacing is 6 to
    12 %).  sqrt(v) ends within a spacing and the spread of the thresholds'
    walk, 25 %, on average over the tensor."""
    torch.manual_seed(0)
    h = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-12, weight_decay=0.0)
    n = 2048
    opts = []
    for bits in (32, 8):
        p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        opts.append((optim.AdamW([p], [g], **h, state_bits=bits), p, g))
    for size in (1e-3, 1e-1, 1e-2):
        for _ in range(3000):
            noise = torch.randn(n, device="cuda") * size
            for opt, p, g in opts:
                g.copy_(noise)
                opt.step()
        v32, v8 = opts[0][0].moments(0)[1].sqrt(), opts[1][0].moments(0)[1].sqrt()
        ratio = (v8 / v32).log()
        assert abs(ratio.mean().item()) < 0.05 and ratio.std().item() < 0.25


def test_state_dict_round_trip(optim):
    g = torch.randn(500, device="cuda")
    a, b = torch.zeros(500, device="cuda"), torch.zeros(500, device="cuda")
    one, two = optim.AdamW([a], [g], **H, state_bits=8), optim.AdamW([b], [g], **H, state_bits=8)
    one.step()
    b.copy_(a)
    two.load_state_dict(one.state_dict())
    one.step()
    two.step()
    assert torch.equal(a, b) and two.steps == 2
    with pytest.raises(ValueError, match="states hold"):
        optim.AdamW([a], [g], state_bits=32).load_state_dict(one.state_dict())


def test_refusals(optim):
    p, g = torch.zeros(10, device="cuda"), torch.zeros(10, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        optim.AdamW([p], [p])
    with pytest.raises(ValueError, match="elements"):
        optim.AdamW([p], [g[:9]])
    with pytest.raises(ValueError, match="dtype"):
        optim.AdamW([p.int()], [g])
    with pytest.raises(ValueError, match="contiguous"):
        optim.AdamW([torch.zeros(10, 2, device="cuda")[:, 0]], [g])
    with pytest.raises(ValueError, match="fp32 parameters"):
        optim.AdamW([p.bfloat16()], [g], copies=[g.bfloat16()])
    with pytest.raises(ValueError, match="state_bits"):
        optim.AdamW([p], [g], state_bits=16)
    with pytest.raises(ValueError, match="contiguous tensor on"):
        optim.AdamW([p], [g.cpu()])
    opt = optim.AdamW([p], [g], lr=float("nan"))
    with pytest.raises(ccl().CclError, match="lr"):
        opt.step()
    assert opt.steps == 0


def test_square_roots_of_every_mantissa(optim):
    """The kernel's square root and quotient are worked out from approximations:
    every mantissa of v at an even and an odd exponent, with random m, gives
    the bits of numpy's correctly rounded ones."""
    v = ((np.uint32(127) << 23) + np.arange(1 << 24, dtype=np.uint32)).view(np.float32)  # 1 .. 4
    m = np.random.default_rng(8).standard_normal(v.size).astype(np.float32)
    z = np.zeros(v.size, np.float32)
    h = dict(lr=0.5, betas=(0.5, 0.5), eps=1e-8, weight_decay=0.0)
    p = torch.zeros(v.size, device="cuda")
    opt = optim.AdamW([p], [torch.zeros_like(p)], **h,
                      states={"exp_avg": [torch.from_numpy(m).cuda()], "exp_avg_sq": [torch.from_numpy(v).cuda()]})
    opt.step()
    np.testing.assert_array_equal(p.cpu().numpy(), adamw.step32(z, z, m, v, 1, **h)[0])


@pytest.mark.parametrize("eps", [1e-8, 0.0, 1e-20])
@pytest.mark.parametrize("bits", [32, 8])
def test_the_ends_of_the_exponent_range(optim, bits, eps):
    """Gradients from subnormal to huge, side by side: numbers outside the fast
    square root's and quotient's range take the exact operations."""
    rng = np.random.default_rng(9)
    g = np.exp2(rng.uniform(-148, 62, 4096)).astype(np.float32) * np.where(rng.random(4096) < 0.5, -1, 1).astype(np.float32)
    g[::7] = 0
    z = np.zeros_like(g)
    h = {**H, "eps": eps}
    p = torch.zeros(g.size, device="cuda")
    opt = optim.AdamW([p], [torch.from_numpy(g).cuda()], **h, state_bits=bits)
    opt.step()
    want, m, v, root = adamw.step32(z, g, z, z, 1, **h)
    np.testing.assert_array_equal(p.cpu().numpy(), want)
    if bits == 8:
        np.testing.assert_array_equal(opt.table.tensors["exp_avg"][0].view(torch.uint8).cpu().numpy(), adamw.encode_m(m)[0])
        np.testing.assert_array_equal(opt.table.tensors["exp_avg_sq"][0].view(torch.uint8).cpu().numpy(), adamw.encode_root(root, v, 1)[0])
    else:
        np.testing.assert_array_equal(opt.moments(0)[0].cpu().numpy(), m)
        np.testing.assert_array_equal(opt.moments(0)[1].cpu().numpy(), v)
