"""Products whose launches have very many workgroups: many experts with wide outputs, rows of one expert only."""

import pytest

import test_gpu_w4 as W
from test_gpu_gated import UACT, UBF, act64, act_of, check, cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_scaled_amd as m
    return m


# 16 passes of 64 rows: 2^21 workgroups; 2^24 of 256 threads, one more than a launch takes, so that 15 share them
@pytest.mark.parametrize("experts,f,rows", [(128, 16384, 970), (256, 65536, 1030)])
def test_w4_passes_of_many_experts(M, experts, f, rows):
    import torch
    k, group, g = 32, 32, experts - 3
    gen = torch.Generator(device="cuda").manual_seed(50)
    codes = torch.randint(0, 256, (experts, 2 * f, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = (torch.rand((experts, 2 * f, 1), generator=gen, device="cuda") * 2.0 ** -6).to(torch.bfloat16)
    packed = M.w4_pack(codes, scales)
    x = W.rows(rows, k, 51)
    splits = [0] * experts
    splits[g] = rows
    h = M.grouped_gated_w4(act_of("swiglu"), splits, x.cuda(), packed)
    # the same rows with that expert's weights alone: the same sums
    alone = M.w4_pack(codes[g:g + 1], scales[g:g + 1])
    assert torch.equal(h, M.grouped_gated_w4(act_of("swiglu"), [rows], x.cuda(), alone))
    # rows at the passes' ends against 64 bits
    some = [0, 63, 64, 959, 960, rows - 1]
    w = [t[g:g + 1].cpu() for t in (codes, scales)] + [None]
    pre, d = W.product64([len(some)], x[some], w, None)
    a, dg, du, mag_a, mag_g = act64("swiglu", pre[:, :f], pre[:, f:])
    tol = 2 * (dg.abs() + mag_g) * d[:, :f] + (pre[:, :f].abs() + 1) * d[:, f:] + UACT * mag_a
    check(h[some], a, tol + UBF * a.abs(), "h")
