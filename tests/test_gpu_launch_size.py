"""Products whose launches have very many workgroups: many experts with wide outputs, rows of one expert only."""

import pytest

import test_gpu_w4 as W
from test_gpu_gated import U32, UACT, UBF, act64, act_of, check, gated64

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


@pytest.mark.parametrize("n,rows", [((1 << 18) - 8, 1), (1 << 18, 20)])
def test_few_bf16_rows_of_many_experts(M, n, rows):
    """2^21 workgroups of 32 weight rows for up to 16 rows, 2^20 of 64 for more."""
    import torch
    experts, k, g = 256, 8, 253
    gen = torch.Generator(device="cuda").manual_seed(52)
    w = torch.randn((experts, n, k), generator=gen, device="cuda", dtype=torch.bfloat16)
    x = W.rows(rows, k, 53)
    splits = [0] * experts
    splits[g] = rows
    got = M.grouped_gemm_bf16("fprop", splits, x.cuda(), w, out_dtype=torch.float32)
    wg = w[g].cpu().double()
    ref, mag = x.double() @ wg.t(), x.double().abs() @ wg.t().abs()
    check(got, ref, (k + 2) * U32 * mag + U32 * ref.abs(), "c")


@pytest.mark.parametrize("f", [1 << 17])
def test_few_gated_rows_of_many_experts(M, f):
    import torch
    experts, k, g, rows = 256, 8, 250, 3
    gen = torch.Generator(device="cuda").manual_seed(54)
    w = torch.randn((experts, 2 * f, k), generator=gen, device="cuda", dtype=torch.bfloat16) * k ** -0.5
    x = W.rows(rows, k, 55)
    splits = [0] * experts
    splits[g] = rows
    h = M.grouped_gated_fwd(act_of("glu"), splits, x.cuda(), w)
    ref, tol, _, _ = gated64("glu", [rows], x, w[g:g + 1].cpu(), None, None)
    check(h, ref, tol + UBF * ref.abs(), "h")
