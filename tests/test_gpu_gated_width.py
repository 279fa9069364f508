"""A gated kind's quantized gradient [gate | up] when the half width is no multiple of 128.  The K step in
which the gate half ends holds row scales of both halves, and the 128-column tile there reaches over the up
half's first columns: both are written by different workgroups, and everything has to arrive."""

import numpy as np
import pytest

import workloads
from oracle import activations
from oracle import quant as Q
from tests.helpers import bf16_f64, compare_quantized, mx_elementwise, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wa", [32, 96, 160, 224, 288])
@pytest.mark.parametrize("kind", ["swiglu", "glu"])
def test_gated_gradient_row_scales(kind, wa):
    import torch
    from moe_grouped_scaled_amd import _native as N
    splits = [64, 0, 37, 130]
    d = workloads.act_case(kind, splits, 2 * wa, seed=wa, std=1.5)
    m, w = int(d["splits"].sum()), 2 * wa
    row = N.QTensor("mxfp8", False, splits, w)
    row.scales.fill_(0xEE)
    N.grouped_scaled_act_bwd(N.act_params(kind), "mxfp8", splits, w, to_dev_bf16(d["x"]), to_dev_bf16(d["dy"]),
                             to_dev(d["p"]), dx_row=row)
    torch.cuda.synchronize()
    dx, _ = activations.scaled_act_bwd(kind, bf16_f64(d["x"]), bf16_f64(d["dy"]), d["p"].astype(np.float64))
    ref = Q.quantize_grouped(dx, splits, "mxfp8", colwise=False)
    scales = row.scales.cpu().numpy()
    compare_quantized("mxfp8", mx_elementwise(row.data.cpu().numpy(), scales, m, w),
                      mx_elementwise(ref["row_data"], ref["row_scales"], m, w))
    if (w // 32) % 4:                                      # unused bytes of a partial last step are zero
        assert not scales.reshape(-1, m, 4)[-1, :, (w // 32) % 4:].any()


@pytest.mark.parametrize("wa", [32, 96, 160, 224, 288])
@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_gated_gradient_columns(fmt, wa):
    import torch
    from moe_grouped_scaled_amd import _native as N
    from oracle import gemm as G
    splits = [64, 0, 37, 130]
    d = workloads.act_case("swiglu", splits, 2 * wa, seed=wa, std=1.5)
    w = 2 * wa
    col = N.QTensor(fmt, True, splits, w)
    amax = torch.empty(len(splits), device="cuda")
    N.grouped_scaled_act_bwd(N.act_params("swiglu"), fmt, splits, w, to_dev_bf16(d["x"]), to_dev_bf16(d["dy"]),
                             to_dev(d["p"]), dx_col=col, dx_group_amax=amax)
    torch.cuda.synchronize()
    dx, _ = activations.scaled_act_bwd("swiglu", bf16_f64(d["x"]), bf16_f64(d["dy"]), d["p"].astype(np.float64))
    ref = Q.quantize_grouped(dx, splits, fmt, rowwise=False)
    gs = col.group_scale.cpu().numpy() if fmt == "nvfp4" else None
    got = G.dequant_col_grouped(fmt, col.data.cpu().numpy(), col.scales.cpu().numpy(), splits, w, gs)
    want = G.dequant_col_grouped(fmt, ref["col_data"], ref["col_scales"], splits, w, ref.get("group_scale"))
    for g, (a, b) in enumerate(zip(got, want)):
        if a.size:   # element for element, but for those next to a rounding border (one in a thousand)
            assert np.mean(np.abs(a - b) > 1e-5 * np.abs(b)) <= 1e-3, g
