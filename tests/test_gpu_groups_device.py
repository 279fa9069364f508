"""Device-resident split sizes that are not on the block's device are refused, and nothing is enqueued."""

import pytest

import test_gpu_w4 as W
from test_gpu_gated import cuda, device_groups
from test_gpu_gated_mlp import params

pytestmark = pytest.mark.gpu


def test_split_sizes_in_host_memory():
    import torch
    import moe_grouped_scaled_amd as M
    from moe_grouped_scaled_amd import _native as N
    w1, w2, b1, b2 = cuda(*params(3, 64, 64, 90, True))
    full = M.GatedMLP("swiglu", w1, w2, b1, b2)
    four = M.W4GatedMLP("swiglu", M.w4_pack(*cuda(*W.weights(3, 128, 64, 32, True, 91))), M.w4_pack(*cuda(*W.weights(3, 64, 64, 32, True, 92))))
    x = torch.ones(8, 64, dtype=torch.bfloat16, device="cuda")
    host = N.DeviceGroups(3, 8, device="cpu")
    for mlp in (full, four):
        with pytest.raises(ValueError, match="the split sizes are on cpu"):
            mlp.forward(x, None, host)
        with pytest.raises(ValueError, match="3 experts"):
            mlp.forward(x, None, device_groups([4, 4], 8))
        with pytest.raises(ValueError, match="capacity"):
            mlp.forward(x, None, device_groups([4, 0, 4], 9))
        with pytest.raises(ValueError, match="GPU"):
            mlp.forward(x.cpu(), None, device_groups([4, 0, 4], 8))
        on = device_groups([4, 0, 4], 8)
        assert torch.equal(mlp.forward(x, None, on)[:4], mlp.forward(x, None, on)[:4])
    torch.cuda.synchronize()
