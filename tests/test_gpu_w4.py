"""Products with 4-bit weights against their formula in 64 bits, the packed layout, and the quantizer.

Bounds: per group of g elements the kernel sums (16 + q) x and (16 + z) x in FP32 (at most 31 |x| each, a rounding a
term at most: 2 (g + 2) 2^-24 31 sum |x|), scales, and adds K / g groups; rounding to BF16 adds 2^-8 of the value.
"""

import math

import pytest

from test_gpu_gated import KINDS, UBF, U32, UACT, LIMIT, act64, act_of, bounds, check, cuda, device_groups

pytestmark = pytest.mark.gpu

SPLITS = {"one_row": [1], "few": [3, 0, 1, 16, 17], "ragged": [0, 70, 33], "empty": [0, 0]}


@pytest.fixture(scope="module")
def M():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_scaled_amd as m
    return m


def weights(e, n, k, group, zeros, seed):
    import torch
    gen = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (e, n, k // 2), generator=gen, dtype=torch.uint8)
    scales = ((torch.rand((e, n, k // group), generator=gen) + 0.1) * 2.0 ** -6).to(torch.bfloat16)
    scales[:, ::5, ::2] *= -1
    z = torch.randint(0, 16, scales.shape, generator=gen, dtype=torch.uint8) if zeros else None
    return codes, scales, z


def values64(codes, scales, zeros):
    import torch
    e, n, kh = codes.shape
    q = torch.stack([codes & 15, codes >> 4], dim=3).view(e, n, 2 * kh).double()
    rep = 2 * kh // scales.shape[2]
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(rep, dim=2)
    return (q - z) * scales.double().repeat_interleave(rep, dim=2)


def product64(splits, x, w, bias):
    """(y, bound before rounding)"""
    import torch
    codes, scales, zeros = w
    v = values64(*w)
    n, k = v.shape[1], v.shape[2]
    group = k // scales.shape[2]
    y = torch.zeros((x.shape[0], n), dtype=torch.float64)
    tol = torch.zeros_like(y)
    for g, at in bounds(splits):
        xd = x[at].double()
        y[at] = xd @ v[g].t()
        xs = xd.abs().view(xd.shape[0], k // group, group).sum(2)
        tol[at] = (2 * (group + 2) + k // group + 4) * U32 * 31 * (xs @ scales[g].double().abs().t())
        if bias is not None:
            y[at] += bias[g].double()
            tol[at] += 2 * U32 * bias[g].double().abs()
    return y, tol + U32 * y.abs()


def rows(m, k, seed):
    import torch
    return torch.randn(m, k, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("group,zeros,n,k", [(128, True, 64, 256), (128, False, 40, 128), (64, True, 17, 192), (64, False, 200, 64),
                                             (32, True, 1, 32), (32, False, 33, 416), (32, True, 96, 1056), (128, True, 30, 1152)])
@pytest.mark.parametrize("split", sorted(SPLITS))
def test_product(M, split, group, zeros, n, k):
    import torch
    splits = SPLITS[split]
    w = weights(len(splits), n, k, group, zeros, seed=n + k)
    x = rows(sum(splits), k, 1)
    bias = rows(len(splits), n, 2)
    packed = M.w4_pack(*cuda(*w))
    assert packed.shape == (len(splits), n, k) and packed.group == group and packed.zeros == zeros
    for b in (None, bias):
        ref, tol = product64(splits, x, w, b)
        for dt, u in ((torch.bfloat16, UBF), (torch.float32, 0.0)):
            y = M.grouped_gemm_w4(splits, x.cuda(), packed, bias=None if b is None else b.cuda(), out_dtype=dt)
            check(y, ref, tol + u * ref.abs(), "y")
            assert torch.equal(y, M.grouped_gemm_w4(splits, x.cuda(), packed, bias=None if b is None else b.cuda(), out_dtype=dt))


@pytest.mark.parametrize("group,zeros,f,k", [(128, True, 64, 256), (64, False, 16, 192), (32, True, 48, 416)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("split", sorted(SPLITS))
def test_gated(M, split, kind, group, zeros, f, k):
    import torch
    splits = SPLITS[split]
    w = weights(len(splits), 2 * f, k, group, zeros, seed=f)
    x, b = rows(sum(splits), k, 3), rows(len(splits), 2 * f, 4)
    p = torch.rand(sum(splits), generator=torch.Generator().manual_seed(5))
    packed = M.w4_pack(*cuda(*w))
    for bias, probs in ((b, p), (None, None)):
        pre, d = product64(splits, x, w, bias)
        a, dg, du, mag_a, mag_g = act64(kind, pre[:, :f], pre[:, f:])
        s = torch.ones(sum(splits), 1, dtype=torch.float64) if probs is None else probs.double()[:, None]
        slope_u = pre[:, :f].clamp(max=LIMIT if kind == "clamped_swiglu" else math.inf).abs() + 1
        tol = s * (2 * (dg.abs() + mag_g) * d[:, :f] + slope_u * d[:, f:] + UACT * mag_a)
        h = M.grouped_gated_w4(act_of(kind), splits, x.cuda(), packed, *cuda(bias, probs))
        check(h, a * s, tol + UBF * (a * s).abs(), "h")


def test_long_reduction_and_wide_output(M):
    import torch
    splits, n, k = [2], 1000, 16384
    w = weights(1, n, k, 128, True, seed=7)
    x = rows(2, k, 8)
    ref, tol = product64(splits, x, w, None)
    y = M.grouped_gemm_w4(splits, x.cuda(), M.w4_pack(*cuda(*w)), out_dtype=torch.float32)
    check(y, ref, tol, "y")


def test_rows_do_not_reach_each_other(M):
    """A row of NaN and infinities, and whatever stands behind the tensors, changes that row only."""
    import torch
    splits, n, k = [3, 18], 40, 96
    w = weights(2, n, k, 32, True, seed=9)
    packed = M.w4_pack(*cuda(*w))
    x = rows(21, k, 10).cuda()
    clean = M.grouped_gemm_w4(splits, x, packed)
    big = torch.full((40, k), math.nan, dtype=torch.bfloat16, device="cuda")
    big[:21] = x
    assert torch.equal(M.grouped_gemm_w4(splits, big[:21], packed), clean)
    for bad in (1, 3, 20):
        z = x.clone()
        z[bad, 5], z[bad, 90] = math.inf, math.nan
        y = M.grouped_gemm_w4(splits, z, packed)
        keep = [i for i in range(21) if i != bad]
        assert torch.equal(y[keep], clean[keep]) and y[bad].isnan().all()


@pytest.mark.parametrize("splits,cap", [([3, 0, 20], 40), ([0, 0], 8), ([60, 0, 0, 2], 62)])
def test_device_resident_split_sizes(M, splits, cap):
    import torch
    f, k, m = 48, 160, sum(splits)
    w = weights(len(splits), 2 * f, k, 32, True, seed=11)
    packed = M.w4_pack(*cuda(*w))
    x = rows(m, k, 12).cuda()
    p = torch.rand(m, device="cuda")
    dg = device_groups(splits, cap)
    wide = lambda t: torch.cat([t, torch.full((cap - m, *t.shape[1:]), math.nan, dtype=t.dtype, device="cuda")])
    h = torch.full((cap, f), 7.0, dtype=torch.bfloat16, device="cuda")
    M.grouped_gated_w4("swiglu", dg, wide(x), packed, probs=wide(p), h=h)
    ref = M.grouped_gated_w4("swiglu", splits, x, packed, probs=p)
    assert (h[m:] == 7).all() and torch.allclose(h[:m].float(), ref.float(), rtol=2 * UBF, atol=1e-4)


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantizer(M, group, zeros):
    """Codes against the rule in 64 bits; an element is off by at most half a step and what rounding the scale to BF16 moves
    the grid's end by."""
    import torch
    gen = torch.Generator().manual_seed(13)
    w = (torch.randn(2, 24, 2 * 128, generator=gen) * 0.05).to(torch.bfloat16)
    w[0, 0] = 0                      # a group of zeros
    w[0, 1] = w[0, 1].abs()          # one-sided groups
    w[0, 2] = -w[0, 2].abs()
    w[0, 3, 5] = 40.0                # an outlier
    w[0, 4] = 1e-38
    codes, scales, z = M.w4_quantize(w.cuda(), group, zeros)
    v = values64(codes.cpu(), scales.cpu(), None if z is None else z.cpu())
    g = w.double().view(2, 24, -1, group)
    lo, hi = g.amin(3).clamp(max=0), g.amax(3).clamp(min=0)
    step = (hi - lo) / 15 if zeros else torch.maximum(hi, -lo) / 7
    s = scales.double().cpu()
    assert ((s - step).abs() <= 2.0 ** -8 * step + 1e-40).all()
    if zeros:
        ref_z = torch.where(s > 0, (-lo / torch.where(s > 0, s, 1.0)).round().clamp(max=15), 0.0)
        assert (z.cpu().double() - ref_z).abs().max() <= 1 and ((z.cpu().double() - ref_z) != 0).double().mean() < 0.01
    # the zero point's own rounding shifts the grid by half a step at most, and the scale's moves its end by 15 x 2^-8 of one
    err = (v.view_as(g) - g).abs()
    assert (err <= (1.0 + 15 * 2.0 ** -8 + 1e-6) * s[..., None] + 1e-37).all()
    assert not v[0, 0].any()


def test_block_and_layer(M):
    """W4GatedMLP against its parts in 64 bits, and inside MoELayer, captured and replayed for other routings."""
    import torch
    e, h, f, tokens, topk = 4, 128, 96, 19, 2
    w1, w2 = weights(e, 2 * f, h, 32, True, 14), weights(e, h, f, 32, False, 15)
    b1, b2 = rows(e, 2 * f, 16), rows(e, h, 17)
    mlp = M.W4GatedMLP("swiglu", M.w4_pack(*cuda(*w1)), M.w4_pack(*cuda(*w2)), *cuda(b1, b2))
    splits = [5, 0, 13, 1]
    x = rows(19, h, 18)
    y = mlp.forward(x.cuda(), None, splits)
    pre, _ = product64(splits, x, w1, b1)
    a = act64("swiglu", pre[:, :f], pre[:, f:])[0]
    ref, _ = product64(splits, a, w2, b2)
    # two roundings to BF16
    assert (y.double().cpu() - ref).norm() <= math.sqrt(2) * UBF * ref.norm()
    with pytest.raises(ValueError, match="no backward"):
        mlp.backward(y)
    layer = M.MoELayer(mlp, topk)
    xd, logits = x.cuda(), torch.randn(tokens, e, device="cuda")

    def layer64():
        top = logits.double().cpu().topk(topk, dim=1)
        wt = torch.softmax(top.values, dim=1)
        out = torch.zeros(tokens, h, dtype=torch.float64)
        v1, v2 = values64(*w1), values64(*w2)
        xx = xd.double().cpu()
        for t in range(tokens):
            for j in range(topk):
                k = int(top.indices[t, j])
                p = v1[k] @ xx[t] + b1[k].double()
                out[t] += wt[t, j] * (v2[k] @ (p[:f] * torch.sigmoid(p[:f]) * p[f:]) + b2[k].double())
        return out

    def near(got):
        ref = layer64()
        assert (got.double().cpu() - ref).norm() <= 2 * UBF * ref.norm()  # three roundings

    near(layer.forward(xd, logits))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(xd, logits)
    for i in range(3):
        xd.copy_(rows(tokens, h, 20 + i))
        logits.copy_(torch.randn(tokens, e, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        near(out)
        assert torch.equal(out, layer.forward(xd, logits))


def test_streams(M):
    import torch
    w = weights(1, 64, 128, 64, True, 30)
    x = rows(3, 128, 31).cuda()
    packed = M.w4_pack(*cuda(*w))
    ref = M.grouped_gemm_w4([3], x, packed)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    assert torch.equal(M.w4_pack(*cuda(*w), stream=side).data, packed.data) if not side.synchronize() else False
    y = M.grouped_gemm_w4([3], x, packed, stream=side)
    side.synchronize()
    assert torch.equal(y, ref)
