"""Device-resident split sizes of another device, expert count or capacity are refused before their offsets are computed: that
computation is a kernel that writes the split sizes' table.  CPU tensors stand in for a GPU's, and those on "meta" for
another one's."""

import contextlib

import pytest
import torch


@pytest.fixture
def blocks(monkeypatch):
    """The two blocks on stand-in tensors, 3 experts, rows of 64."""
    import moe_grouped_scaled_amd as M
    from moe_grouped_scaled_amd import gated, w4
    monkeypatch.setattr(gated, "_check", lambda what, t, *a, **k: t)
    monkeypatch.setattr(w4, "_check", lambda what, t, *a, **k: t)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    full = M.GatedMLP("swiglu", torch.zeros(3, 128, 64, dtype=torch.bfloat16), torch.zeros(3, 64, 64, dtype=torch.bfloat16))
    data = torch.zeros(3 * 8 * (1024 + 64), dtype=torch.uint8)
    four = M.W4GatedMLP("swiglu", M.W4Tensor(data, (3, 128, 64), 64, False), M.W4Tensor(data[:3 * 4 * (1024 + 64)], (3, 64, 64), 64, False))
    return [full, four]


def groups(experts, rows, device):
    from moe_grouped_scaled_amd import _native as N
    g = N.DeviceGroups(experts, rows, device=device)

    def update(stream=None):
        raise AssertionError("the offsets' computation was enqueued")

    g.update = update
    return g


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("experts,rows,device,match", [(3, 8, "meta", "the split sizes are on meta"), (2, 8, "cpu", "3 experts"),
                                                       (3, 9, "cpu", "capacity")])
def test_refused_before_the_update(blocks, which, experts, rows, device, match):
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=match):
        blocks[which].forward(x, None, groups(experts, rows, device))


@pytest.mark.parametrize("which", [0, 1])
def test_right_ones_are_updated(blocks, which):
    with pytest.raises(AssertionError, match="was enqueued"):
        blocks[which].forward(torch.zeros(8, 64, dtype=torch.bfloat16), None, groups(3, 8, "cpu"))
