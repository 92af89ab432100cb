"""Calls that have nothing to write: no-ops, also without a GPU."""
from __future__ import annotations

import pytest
import torch

from test_experts_abi import at, lib, ptrs, sizes  # noqa: F401 (lib is a fixture)


def test_rows_without_a_place_to_go(lib):  # noqa: F811
    """Tokens whose rank's buffer holds no rows, as where all their experts are on
    other ranks: nothing is written and nothing is refused."""
    f = lib.LIB.ccl_moe_to_experts
    x, rows, null = ptrs(at(0)), ptrs(at(1)), ptrs(0)
    for hidden, dt in ((64, 1), (63, 1), (64, 0), (1, 0)):
        assert f(x, rows, sizes(10), 1, 2, hidden, dt, null, sizes(0), None) == lib.CCL_OK, lib.ccl_last_error()
    x2, rows2, null2 = ptrs(at(0), 0), ptrs(at(1), 0), ptrs(0, at(2))
    assert f(x2, rows2, sizes(10, 0), 2, 2, 64, 1, null2, sizes(0, 20), None) == lib.CCL_OK, lib.ccl_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hidden", [64, 63, 7])
def test_a_rank_whose_tokens_all_go_elsewhere(lib, hidden, dtype):  # noqa: F811
    """The whole local half on one such rank: zeros come back."""
    T, k, E, n = 5, 2, 4, 24
    ids = [torch.full((T, k), 99, dtype=torch.int32, device="cuda")]
    offsets, rows = [torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")], [torch.empty_like(ids[0])]
    lib.ccl_moe_sort(ids, E, offsets, rows)
    assert (offsets[0] == 0).all() and (rows[0] == -1).all()
    x = [torch.randn(T, hidden, device="cuda").to(dtype)]
    none = [torch.empty(0, hidden, dtype=dtype, device="cuda")]
    lib.ccl_moe_to_experts(x, rows, none)
    out, gates = [torch.full((T, hidden), 7.0, device="cuda").to(dtype)], [torch.rand(T, k, device="cuda")]
    lib.ccl_moe_from_experts(none, rows, gates, out)
    dgates = [torch.full((T, k), 7.0, device="cuda")]
    lib.ccl_moe_from_experts_grad(x, none, rows, gates, [torch.empty_like(none[0])], dgates)
    assert (out[0] == 0).all() and (dgates[0] == 0).all()
    if dtype == torch.bfloat16:
        w, dw = [torch.randn(E, n, hidden, device="cuda").to(dtype)], [torch.full((E, n, hidden), 7.0, device="cuda")]
        y = [torch.empty(0, n, dtype=dtype, device="cuda")]
        lib.ccl_moe_product(none, offsets, w, y)
        lib.ccl_moe_product_grad_input(y, offsets, w, none)
        lib.ccl_moe_product_grad_weight(y, none, offsets, dw)
        assert (dw[0] == 0).all()
