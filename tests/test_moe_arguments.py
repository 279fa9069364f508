"""Arguments of the routing calls at the ends of their types: sizes that do not fit their C arguments are refused, not
cut to their lower 32 bits; every finite factor on the weights is taken."""

import pytest


@pytest.mark.parametrize("n", [(1 << 32) + 2, 1 << 31, -1, -(1 << 32) + 2])
def test_counts_beyond_32_bits(n):
    import torch
    import moe_grouped_scaled_amd as M
    from moe_grouped_scaled_amd.moe import moe_dispatch_workspace_bytes
    with pytest.raises(ValueError, match="topk"):
        M.moe_route(torch.zeros(4, 8), n)
    with pytest.raises(ValueError, match="num_experts"):
        M.moe_dispatch(torch.zeros((4, 2), dtype=torch.int32), n)
    with pytest.raises(ValueError, match="num_experts"):
        moe_dispatch_workspace_bytes(4000, 2, n)
    with pytest.raises(ValueError, match="topk"):
        moe_dispatch_workspace_bytes(4000, n, 8)
    assert moe_dispatch_workspace_bytes(4000, 2, 8) > 0


def test_every_finite_scale():
    from test_moe import _lib, _refused
    N, lib = _lib()
    largest = float(2.0 ** 128 - 2.0 ** 104)
    call = lambda scale: lib.mgs_moe_route(N.RouteParams(0, 1, scale), 0, 8, 2, None, 0, 8, None, None, None)
    for scale in (largest, -largest, 3.4e38, -3.4e38, 2.0 ** -149, 0.0):
        assert call(scale) == 0, scale
    for scale in (float("inf"), -float("inf"), float("nan")):
        _refused(-1, call(scale), "finite")
