"""Host-side refusals of the router's and the layer norm's entry points (no GPU: nothing here is launched)."""
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


def at(i, r=0):
    return BASE + (i << 32) + (r << 26)


def one(i):
    return ptrs(at(i))


def two(i):
    return ptrs(at(i), at(i, 1))


GATE = dict(logits=one(0), tokens=sizes(10), p=1, k=2, e=8, dt=0, score=0, norm=1, scale=1.0, ids=one(1), gates=one(2), together=0,
            counts=one(3), losses=one(4), ws=at(5), ws_bytes=1 << 24)


def gate(lib, **kw):
    a = {**GATE, **kw}
    return lib.LIB.ccl_moe_gate(*[a[n] for n in GATE], None)


@pytest.mark.parametrize("change", [
    dict(p=0), dict(p=65), dict(k=0), dict(k=17, e=64), dict(k=9), dict(e=0), dict(e=1025), dict(tokens=None), dict(tokens=sizes(2 ** 31)),
    dict(dt=7), dict(score=2), dict(score=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(logits=None), dict(logits=ptrs(0)),
    dict(logits=ptrs(at(0) + 2)), dict(ids=None), dict(gates=ptrs(at(2) + 1)), dict(gates=None), dict(counts=None), dict(losses=None),
    dict(ws=None), dict(ws=at(5) + 4), dict(ws_bytes=100), dict(ids=ptrs(at(0) + 8)), dict(gates=ptrs(at(1) + 4)), dict(losses=ptrs(at(3) + 32)),
    dict(ws=at(0)), dict(counts=ptrs(0)),
    dict(p=2, logits=two(0), tokens=sizes(10, 10), ids=ptrs(at(1), at(1) + 8), gates=two(2), counts=two(3), losses=two(4)),
    dict(p=2, logits=two(0), tokens=sizes(2 ** 29, 2 ** 29), together=1, ids=two(1), gates=two(2), counts=two(3), losses=two(4)),
], ids=lambda c: ",".join(c))
def test_gate_refusals(lib, change):
    assert gate(lib, **change) == lib.CCL_ERR_INVALID_ARG
    assert lib.ccl_last_error()


def test_integer_logits_are_unsupported(lib):
    assert gate(lib, dt=2) == lib.CCL_ERR_UNSUPPORTED


BALANCE = dict(logits=one(0), ids=one(1), tokens=sizes(10), p=1, k=2, e=8, dt=0, score=0, together=0, counts=one(3), losses=one(4), ws=at(5),
               ws_bytes=1 << 24)


@pytest.mark.parametrize("change", [
    dict(p=0), dict(k=9), dict(ids=None), dict(ids=ptrs(at(1) + 2)), dict(counts=None), dict(losses=None), dict(ws=None), dict(ws_bytes=8),
    dict(counts=ptrs(at(1))), dict(losses=ptrs(at(0))), dict(score=5), dict(logits=None),
], ids=lambda c: ",".join(c))
def test_balance_refusals(lib, change):
    a = {**BALANCE, **change}
    assert lib.LIB.ccl_moe_balance(*[a[n] for n in BALANCE], None) == lib.CCL_ERR_INVALID_ARG


GATE_GRAD = dict(logits=one(0), ids=one(1), dgates=one(2), tokens=sizes(10), p=1, k=2, e=8, dt=0, score=0, norm=1, scale=1.0, counts=one(3),
                 dlosses=one(4), bscale=1.0, dlogits=one(6))


@pytest.mark.parametrize("change", [
    dict(p=65), dict(k=0), dict(dgates=None), dict(ids=None), dict(dlogits=None), dict(dlogits=one(0)), dict(dlogits=ptrs(at(1) + 4)),
    dict(counts=None), dict(bscale=float("nan")), dict(dgates=ptrs(0)), dict(counts=ptrs(0)), dict(dlosses=ptrs(at(4) + 1)), dict(dlogits=one(3)),
], ids=lambda c: ",".join(c))
def test_gate_gradient_refusals(lib, change):
    a = {**GATE_GRAD, **change}
    assert lib.LIB.ccl_moe_gate_grad(*[a[n] for n in GATE_GRAD], None) == lib.CCL_ERR_INVALID_ARG


def test_balance_gradient_refusals(lib):
    def call(**kw):
        a = dict(logits=one(0), counts=one(3), dlosses=one(4), tokens=sizes(10), p=1, k=2, e=8, dt=1, score=1, scale=1.0, dlogits=one(6))
        a.update(kw)
        return lib.LIB.ccl_moe_balance_grad(*a.values(), None)

    for kw in (dict(counts=None), dict(counts=ptrs(0)), dict(scale=float("inf")), dict(dlogits=one(0)), dict(k=9), dict(p=0), dict(dt=9)):
        assert call(**kw) == lib.CCL_ERR_INVALID_ARG, kw


NORM = dict(x=one(0), residual=one(1), weight=one(2), bias=one(3), rows=sizes(10), p=1, cols=64, eps=1e-5, dt=1, wt=0, y=one(4), sum=one(5),
            mean=one(6), rstd=one(7))


@pytest.mark.parametrize("change", [
    dict(p=0), dict(p=65), dict(cols=0), dict(rows=None), dict(rows=sizes(2 ** 31)), dict(eps=-1.0), dict(eps=float("nan")), dict(dt=5), dict(wt=5),
    dict(residual=None), dict(sum=None), dict(mean=None), dict(rstd=None), dict(x=None), dict(weight=None), dict(y=None), dict(x=ptrs(at(0) + 1)),
    dict(weight=ptrs(at(2) + 2)), dict(y=one(0)), dict(y=ptrs(at(1) + 128)), dict(sum=ptrs(at(4) + 16)), dict(sum=one(1)), dict(mean=ptrs(at(7) + 4)),
    dict(y=ptrs(at(2))), dict(rstd=ptrs(0)), dict(bias=ptrs(0)),
], ids=lambda c: ",".join(c))
def test_norm_refusals(lib, change):
    a = {**NORM, **change}
    assert lib.LIB.ccl_layer_norm(*a.values(), None) == lib.CCL_ERR_INVALID_ARG
    assert lib.ccl_last_error()


NORM_GRAD = dict(dy=one(0), dsum=one(1), x=one(2), weight=one(3), mean=one(4), rstd=one(5), rows=sizes(10), p=1, cols=64, dt=1, wt=0, dx=one(6), dwt=0,
                 dweight=one(7), dbias=one(8), ws=at(9), ws_bytes=1 << 24)


@pytest.mark.parametrize("change", [
    dict(p=0), dict(cols=0), dict(dwt=7), dict(dx=None), dict(mean=None), dict(rstd=ptrs(at(5) + 2)), dict(dy=ptrs(0)), dict(dx=one(0)), dict(dx=one(1)),
    dict(dweight=one(3)), dict(dbias=one(7)), dict(ws=None), dict(ws_bytes=64), dict(ws=at(9) + 8), dict(ws=at(6)), dict(dweight=ptrs(at(7) + 2)),
    dict(p=2, dy=two(0), dsum=two(1), x=two(2), weight=two(3), mean=two(4), rstd=two(5), rows=sizes(10, 0), dx=two(6), dweight=ptrs(at(7), at(7)),
         dbias=two(8)),
], ids=lambda c: ",".join(c))
def test_norm_gradient_refusals(lib, change):
    a = {**NORM_GRAD, **change}
    assert lib.LIB.ccl_layer_norm_grad(*a.values(), None) == lib.CCL_ERR_INVALID_ARG


def test_unsupported_and_empty_calls(lib):
    assert lib.LIB.ccl_layer_norm(*{**NORM, "cols": 16385}.values(), None) == lib.CCL_ERR_UNSUPPORTED
    assert lib.LIB.ccl_layer_norm(*{**NORM, "dt": 2}.values(), None) == lib.CCL_ERR_UNSUPPORTED
    nothing = {**NORM, "rows": sizes(0), **{n: ptrs(0) for n in ("x", "residual", "weight", "bias", "y", "sum", "mean", "rstd")}}
    assert lib.LIB.ccl_layer_norm(*nothing.values(), None) == lib.CCL_OK
    g = {**NORM_GRAD, "rows": sizes(0), "dweight": None, "dbias": None, "ws": None, "ws_bytes": 0}
    assert lib.LIB.ccl_layer_norm_grad(*g.values(), None) == lib.CCL_OK
    assert gate(lib, tokens=sizes(0), counts=None, losses=None) == lib.CCL_OK
    assert lib.LIB.ccl_moe_gate_grad(*{**GATE_GRAD, "tokens": sizes(0)}.values(), None) == lib.CCL_OK


def test_workspace_sizes(lib):
    assert lib.ccl_moe_balance_workspace_bytes(0, 8) == lib.ccl_moe_balance_workspace_bytes(1, 0) == lib.ccl_moe_balance_workspace_bytes(65, 8) == 0
    assert lib.ccl_moe_balance_workspace_bytes(1, 1025) == 0 and lib.ccl_moe_balance_workspace_bytes(64, 1024) > 0
    assert lib.ccl_layer_norm_grad_workspace_bytes(1, 0) == lib.ccl_layer_norm_grad_workspace_bytes(1, 16385) == 0
    assert lib.ccl_layer_norm_grad_workspace_bytes(64, 16384) > 0
