"""Every form of the kernels for few rows, and of the larger tiles with what their epilogues take, at small sizes.

Which form runs goes by the rows of a group and by how many workgroups there are: a wide output with a short reduction
reaches those that large weights take.  References and bounds are those of `test_gpu_gated` and `test_gpu_w4`.
"""

import math

import pytest

import test_gpu_w4 as W
from test_gpu_gated import (HALVES, KINDS, LARGE, U32, UACT, UBF, LIMIT, act64, act_of, check, check_backward, check_pre, cuda,
                            device_groups, gated64, gated_case, normal, operands, product64)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_scaled_amd as m
    return m


# ------------------------------------------------------------------------------------------------- few BF16 rows

# 16, 32 and 64 rows of a workgroup
FEW = [[1, 0], [16, 3], [17, 32], [31, 0], [64, 5], [0, 48]]
WIDE = 8200  # two experts: 514 workgroups of 32 weight rows


@pytest.mark.parametrize("n", [40, WIDE])
@pytest.mark.parametrize("k", [8, 200, 584])
@pytest.mark.parametrize("splits", FEW)
def test_few_rows(M, splits, n, k):
    import torch
    a, b = operands("fprop", splits, n, k, seed=n + k)
    bias = normal(torch.Generator().manual_seed(1), 2, n)
    c = torch.randn(sum(splits), n, generator=torch.Generator().manual_seed(2))
    for bs in (None, bias):
        ref, mag = product64("fprop", splits, a, b, bs)
        ag, bg, bsg = cuda(a, b, bs)
        for dt, u in ((torch.bfloat16, UBF), (torch.float32, U32)):
            got = M.grouped_gemm_bf16("fprop", splits, ag, bg, bias=bsg, out_dtype=dt)
            check(got, ref, (k + 2) * U32 * mag + u * ref.abs(), "c")
        got = M.grouped_gemm_bf16("fprop", splits, ag, bg, c.cuda(), bias=bsg, accumulate=True)
        check(got, ref + c.double(), (k + 3) * U32 * mag + 2 * U32 * (ref.abs() + c.double().abs()), "accumulated")


@pytest.mark.parametrize("f", [40, 4104])
@pytest.mark.parametrize("k", [8, 200])
@pytest.mark.parametrize("splits", FEW)
@pytest.mark.parametrize("kind", KINDS)
def test_few_rows_gated(M, kind, splits, f, k):
    import torch
    x, w, b, p = gated_case(kind, splits, f, k, seed=f)
    ref, tol, pre, dpre = gated64(kind, splits, x, w, b, p)
    xg, wg, bg, pg = cuda(x, w, b, p)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.full((sum(splits), 2 * f), math.nan, dtype=dt, device="cuda")
        h = M.grouped_gated_fwd(act_of(kind), splits, xg, wg, bg, pg, pre=out)
        check(h, ref, tol + UBF * ref.abs(), "h")
        check_pre(out, pre, dpre, kind, f)


@pytest.mark.parametrize("n", [40, WIDE])
@pytest.mark.parametrize("splits,cap", [([90, 1, 0, 0, 0, 0, 0, 3], 100), ([0, 0, 0, 0, 0, 0, 0, 33], 40), ([3, 0], 8)])
def test_few_rows_of_a_capacity(M, splits, cap, n):
    """Device-resident split sizes: a group of more rows than the capacity lets expect is read in several passes."""
    import torch
    k, m = 136, sum(splits)
    a, b = operands("fprop", splits, n, k, seed=31)
    ref, mag = product64("fprop", splits, a, b)
    wide = torch.cat([a, torch.full((cap - m, k), math.nan, dtype=torch.bfloat16)]).cuda()
    c = torch.full((cap, n), 7.0, device="cuda")
    M.grouped_gemm_bf16("fprop", device_groups(splits, cap), wide, b.cuda(), c)
    check(c[:m], ref, (k + 2) * U32 * mag + U32 * ref.abs(), "c")
    assert (c[m:] == 7).all()


# -------------------------------------------------------------------------------------------------- larger tiles


@pytest.mark.parametrize("mode,splits,n,k", LARGE)
def test_bias_and_accumulate_on_larger_tiles(M, mode, splits, n, k):
    import torch
    a, b = operands(mode, splits, n, k, seed=32)
    bias = None if mode == "wgrad" else normal(torch.Generator().manual_seed(33), len(splits), n)
    ref, mag = product64(mode, splits, a, b, bias)
    length = max(splits) if mode == "wgrad" else k
    ag, bg, bias_g = cuda(a, b, bias)
    if bias is not None:
        for dt, u in ((torch.bfloat16, UBF), (torch.float32, U32)):
            got = M.grouped_gemm_bf16(mode, splits, ag, bg, bias=bias_g, out_dtype=dt)
            check(got, ref, (length + 2) * U32 * mag + u * ref.abs(), "c")
    c = torch.randn(ref.shape, generator=torch.Generator().manual_seed(34))
    got = M.grouped_gemm_bf16(mode, splits, ag, bg, c.cuda(), bias=bias_g, accumulate=True)
    check(got, ref + c.double(), (length + 3) * U32 * mag + 2 * U32 * (ref.abs() + c.double().abs()), "accumulated")


TILES = [([100, 300, 0, 77], 3200, 40), ([1000, 500], 4096 - 8, 72), (HALVES[1], 3200, 136)]


@pytest.mark.parametrize("splits,f,k", TILES)
@pytest.mark.parametrize("kind", ["clamped_swiglu", "glu"])
def test_gated_kinds_on_larger_tiles(M, kind, splits, f, k):
    import torch
    x, w, b, p = gated_case(kind, splits, f, k, seed=35)
    ref, tol, pre, dpre = gated64(kind, splits, x, w, b, p)
    xg, wg, bg, pg = cuda(x, w, b, p)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.empty((sum(splits), 2 * f), dtype=dt, device="cuda")
        h = M.grouped_gated_fwd(act_of(kind), splits, xg, wg, bg, pg, pre=out)
        check(h, ref, tol + UBF * ref.abs(), "h")
        check_pre(out, pre, dpre, kind, f)
        check_backward(M, kind, splits, 2 * f, k, seed=36, probs=True, pre_dtype=dt)


@pytest.mark.parametrize("splits,cap", [([100, 0, 300, 7], 500), ([1000, 0, 500, 0], 1600), ([0, 0, 0, 0], 300)])
@pytest.mark.parametrize("n,k", [(72, 136), (4096 - 8, 72)])
def test_dgrad_of_device_resident_split_sizes(M, splits, cap, n, k):
    """The rows that there are, against 64 bits; the others stay as they are."""
    import torch
    m = sum(splits)
    a, b = operands("dgrad", splits, n, k, seed=37)
    ref, mag = product64("dgrad", splits, a, b)
    wide = torch.cat([a, torch.full((cap - m, k), math.nan, dtype=torch.bfloat16)]).cuda()
    for dt, u in ((torch.bfloat16, UBF), (torch.float32, U32)):
        c = torch.full((cap, n), 7.0, dtype=dt, device="cuda")
        M.grouped_gemm_bf16("dgrad", device_groups(splits, cap), wide, b.cuda(), c)
        check(c[:m], ref, (k + 2) * U32 * mag + u * ref.abs(), "c")
        assert (c[m:] == 7).all()


# ------------------------------------------------------------------------------------------------- 4-bit weights

# rows of a pass: 4, 16, 32, 64, and several passes
W4_ROWS = [[4, 1], [16, 9], [32, 20], [64, 40], [150, 0]]
PACKED = [(128, True, 384), (128, False, 128), (64, True, 192), (64, False, 64), (32, True, 160), (32, False, 416)]


@pytest.mark.parametrize("group,zeros,k", PACKED)
@pytest.mark.parametrize("n", [40, 4100, 16391])  # few, some and many blocks of 16 weight rows of two experts
def test_w4_forms(M, n, group, zeros, k):
    import torch
    w = W.weights(2, n, k, group, zeros, seed=38)
    packed = M.w4_pack(*cuda(*w))
    bias = W.rows(2, n, 39)
    for splits in W4_ROWS:
        x = W.rows(sum(splits), k, 40)
        ref, tol = W.product64(splits, x, w, bias)
        for dt, u in ((torch.bfloat16, UBF), (torch.float32, 0.0)):
            y = M.grouped_gemm_w4(splits, x.cuda(), packed, bias=bias.cuda(), out_dtype=dt)
            check(y, ref, tol + u * ref.abs(), "y %s" % splits)


@pytest.mark.parametrize("group,zeros,k", PACKED)
@pytest.mark.parametrize("f", [48, 8208])
def test_w4_gated_forms(M, f, group, zeros, k):
    import torch
    w = W.weights(2, 2 * f, k, group, zeros, seed=41)
    packed = M.w4_pack(*cuda(*w))
    bias = W.rows(2, 2 * f, 42)
    for splits, kind in zip(W4_ROWS, ("swiglu", "clamped_swiglu", "glu", "clamped_swiglu", "swiglu")):
        x, p = W.rows(sum(splits), k, 43), torch.rand(sum(splits), generator=torch.Generator().manual_seed(44))
        pre, d = W.product64(splits, x, w, bias)
        a, dg, du, mag_a, mag_g = act64(kind, pre[:, :f], pre[:, f:])
        s = p.double()[:, None]
        slope_u = pre[:, :f].clamp(max=LIMIT if kind == "clamped_swiglu" else math.inf).abs() + 1
        tol = s * (2 * (dg.abs() + mag_g) * d[:, :f] + slope_u * d[:, f:] + UACT * mag_a)
        h = M.grouped_gated_w4(act_of(kind), splits, x.cuda(), packed, *cuda(bias, p))
        check(h, a * s, tol + UBF * (a * s).abs(), "h %s" % splits)


def test_w4_pack_on_a_stream(M):
    """Packed on a stream of its own, waited for, then compared."""
    import torch
    w = cuda(*W.weights(1, 64, 128, 64, True, 45))
    packed = M.w4_pack(*w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = M.w4_pack(*w, stream=side)
    side.synchronize()
    assert torch.equal(got.data, packed.data)
