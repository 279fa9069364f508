"""Norms past FP32's range: returned as infinity, while the gradients are scaled by the FP64 norm's factor.

The factor is rounded to FP32: half a step, 2^-24 of it, or 2^-150 where it is subnormal; the product and a BF16 output are
rounded once each.
"""

import math

import pytest

from test_gpu_grad_clip import EPS, norm64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["same", "bf16"])
@pytest.mark.parametrize("max_norm", [1000.0, 1.0])
def test_norm_past_fp32(max_norm, out):
    import torch
    import moe_grouped_scaled_amd as M
    gen = torch.Generator().manual_seed(95)
    host = [(torch.rand(n, generator=gen) + 1.0) * 1e38 for n in (300, 2051, 7)]
    ref = norm64(host)
    assert 3.5e38 < ref < 1e40
    dev = [t.cuda() for t in host]
    dst = None if out == "same" else [torch.empty(t.shape, dtype=torch.bfloat16, device="cuda") for t in host]
    assert M.grad_norm(dev).item() == math.inf
    assert M.clip_grad_norm(dev, max_norm, eps=EPS, out=dst).item() == math.inf
    scale = max_norm / (ref + EPS)
    u = 2.0 ** -150 / scale + 2 * 2.0 ** -24 + (2.0 ** -8 if out == "bf16" else 0.0)
    for got, src in zip(dst or dev, host):
        want = src.double() * scale
        assert ((got.double().cpu() - want).abs() <= 1.01 * u * want).all()
