"""Sizes of the routing calls that do not fit their C arguments are refused, not cut to their lower 32 bits."""

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
