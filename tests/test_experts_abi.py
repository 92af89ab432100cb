"""Host-side refusals of the experts' and AdamW entry points (no GPU: nothing here is launched)."""
from __future__ import annotations

import ctypes

import pytest

BASE = 0x7F0000000000  # fake device addresses: never dereferenced by a rejected call


@pytest.fixture(scope="module")
def lib():
    from a2a_ring_ordered_gb300 import build

    build.build()
    from a2a_ring_ordered_gb300 import ccl

    return ccl


def ptrs(*v):
    return (ctypes.c_void_p * len(v))(*v)


def sizes(*v):
    return (ctypes.c_size_t * len(v))(*v)


def at(i):
    return BASE + (i << 24)


def test_sort_refusals(lib):
    f = lib.LIB.ccl_moe_sort
    ok = dict(ids=ptrs(at(0)), tokens=sizes(10), p=1, k=2, e=4, off=ptrs(at(1)), rows=ptrs(at(2)))

    def call(**kw):
        a = {**ok, **kw}
        return f(a["ids"], a["tokens"], a["p"], a["k"], a["e"], None, a["off"], a["rows"], None)

    for kw in (dict(p=0), dict(p=65), dict(k=0), dict(k=17), dict(e=0), dict(e=1025), dict(tokens=None), dict(off=None),
               dict(ids=None), dict(rows=ptrs(0)), dict(ids=ptrs(at(0) + 2)), dict(tokens=sizes(2 ** 31)),
               dict(rows=ptrs(at(0) + 4)), dict(off=ptrs(at(2) + 4))):
        assert call(**kw) == lib.CCL_ERR_INVALID_ARG, kw
        assert lib.ccl_last_error()


def test_rows_refusals(lib):
    to, back, grad = lib.LIB.ccl_moe_to_experts, lib.LIB.ccl_moe_from_experts, lib.LIB.ccl_moe_from_experts_grad
    n, cap = sizes(10), sizes(20)
    x, rows, y, w = ptrs(at(0)), ptrs(at(1)), ptrs(at(2)), ptrs(at(3))
    bad, unsupported = lib.CCL_ERR_INVALID_ARG, lib.CCL_ERR_UNSUPPORTED
    assert to(x, rows, n, 1, 2, 0, 1, y, cap, None) == bad                     # hidden 0
    assert to(x, rows, n, 1, 2, 64, 2, y, cap, None) == unsupported           # int32 rows
    assert to(x, rows, n, 1, 2, 64, 9, y, cap, None) == bad
    assert to(x, rows, n, 1, 2, 64, 1, y, None, None) == bad
    assert to(x, rows, n, 1, 2, 64, 1, ptrs(at(0) + 128), cap, None) == bad     # sorted over x
    assert to(ptrs(at(0) + 1), rows, n, 1, 2, 64, 1, y, cap, None) == bad
    assert to(None, rows, n, 1, 2, 64, 1, y, cap, None) == bad
    assert back(y, cap, rows, w, n, 1, 2, 64, 1, ptrs(at(2)), None) == bad      # out over y
    assert back(y, cap, rows, ptrs(0), n, 1, 2, 64, 1, x, None) == bad
    assert back(y, None, rows, w, n, 1, 2, 64, 1, x, None) == bad
    assert grad(x, None, cap, rows, w, n, 1, 2, 64, 1, y, ptrs(at(4)), None) == bad  # dweights without y
    assert grad(x, y, cap, rows, w, n, 1, 2, 64, 1, y, ptrs(at(4)), None) == bad  # dy over y
    assert grad(x, y, cap, rows, w, n, 1, 2, 64, 1, None, ptrs(at(3)), None) == bad  # dweights over weights


def test_empty_calls_are_no_ops(lib):
    n0 = sizes(0, 0)
    null = ptrs(0, 0)
    assert lib.LIB.ccl_moe_to_experts(null, null, n0, 2, 2, 64, 1, null, n0, None) == lib.CCL_OK
    assert lib.LIB.ccl_moe_from_experts(null, n0, null, None, n0, 2, 2, 64, 0, null, None) == lib.CCL_OK
    assert lib.LIB.ccl_moe_from_experts_grad(null, null, n0, null, None, n0, 2, 2, 64, 0, null, None, None) == lib.CCL_OK
    assert lib.LIB.ccl_moe_product(null, null, null, n0, 2, 4, 64, 64, null, None) == lib.CCL_OK
    hyper = lib.AdamWHyper(1e-3, 0.9, 0.99, 1e-8, 0.0, 1, None)
    assert lib.LIB.ccl_adamw_step(None, 0, 0, 1, 32, ctypes.byref(hyper), None) == lib.CCL_OK
    empty = (lib.AdamWTensor * 2)()
    assert lib.LIB.ccl_adamw_step(empty, 2, 0, 1, 32, ctypes.byref(hyper), None) == lib.CCL_OK


def test_product_refusals(lib):
    f, gw = lib.LIB.ccl_moe_product, lib.LIB.ccl_moe_product_grad_weight
    x, o, w, y, n = ptrs(at(0)), ptrs(at(1)), ptrs(at(2)), ptrs(at(3)), sizes(8)
    bad = lib.CCL_ERR_INVALID_ARG
    for args in ((x, o, w, n, 0, 4, 64, 64, y), (x, o, w, n, 65, 4, 64, 64, y), (x, o, w, n, 1, 0, 64, 64, y),
                 (x, o, w, n, 1, 1025, 64, 64, y), (x, o, w, n, 1, 4, 0, 64, y), (x, o, w, n, 1, 4, 64, 2 ** 22 + 1, y),
                 (x, o, w, sizes(2 ** 31), 1, 4, 64, 64, y), (x, None, w, n, 1, 4, 64, 64, y), (None, o, w, n, 1, 4, 64, 64, y),
                 (ptrs(at(0) + 1), o, w, n, 1, 4, 64, 64, y), (x, ptrs(at(1) + 2), w, n, 1, 4, 64, 64, y),
                 (x, o, w, n, 1, 4, 64, 64, ptrs(at(2) + 64)), (x, o, w, n, 1, 4, 64, 64, ptrs(at(0)))):
        assert f(*args, None) == bad, args
    assert gw(x, y, o, n, 1, 4, 64, 64, 2, w, None) == lib.CCL_ERR_UNSUPPORTED
    assert gw(x, y, o, n, 1, 4, 64, 64, 0, ptrs(at(2) + 2), None) == bad  # fp32 at a 2-byte address


def test_adamw_refusals(lib):
    def entry(**kw):
        e = dict(param=at(0), grad=at(1), exp_avg=at(2), exp_avg_sq=at(3), exp_avg_scale=at(4), exp_avg_sq_scale=at(5),
                 copy=0, n=100)
        e.update(kw)
        t = (lib.AdamWTensor * 1)()
        for k, v in e.items():
            setattr(t[0], k, v)
        return t

    good = (1e-3, 0.9, 0.99, 1e-8, 0.01, 1, None)

    def call(t=None, count=1, pdt=0, gdt=1, bits=8, hyper=good):
        return lib.LIB.ccl_adamw_step(t if t is not None else entry(), count, pdt, gdt, bits,
                                      None if hyper is None else ctypes.byref(lib.AdamWHyper(*hyper)), None)

    bad = lib.CCL_ERR_INVALID_ARG
    assert call(pdt=2) == bad and call(gdt=7) == bad and call(bits=16) == bad and call(hyper=None) == bad
    for i, v in ((0, -1.0), (0, float("inf")), (1, 1.0), (1, -0.1), (2, 1.0), (2, float("nan")), (3, -1e-8), (4, -1.0), (5, 0)):
        h = list(good)
        h[i] = v
        assert call(hyper=h) == bad, (i, v)
    assert call(hyper=good[:6] + (BASE + 2,)) == bad
    for kw in (dict(param=0), dict(grad=at(1) + 1), dict(exp_avg=0), dict(exp_avg_scale=0), dict(exp_avg_sq_scale=at(5) + 2),
               dict(grad=at(0) + 4), dict(copy=at(1)), dict(copy=at(6) + 1), dict(n=2 ** 42)):
        assert call(entry(**kw)) == bad, kw
        assert "tensor 0" in lib.ccl_last_error()
    assert call(entry(copy=at(6)), pdt=1) == bad  # a copy beside bf16 parameters
    assert lib.LIB.ccl_adamw_step(None, 1, 0, 1, 32, ctypes.byref(lib.AdamWHyper(*good)), None) == bad
