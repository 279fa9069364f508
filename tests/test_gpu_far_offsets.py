"""Tensors of more than 2^31 elements: the rows, columns and groups behind that, and around it, against 64 bits."""

import pytest

from test_gpu_gated import UBF, U32, UACT, act64
from test_gpu_w4 import values64, weights

pytestmark = pytest.mark.gpu

WIDE = 8192


@pytest.fixture(scope="module")
def M():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_scaled_amd as m
    yield m
    torch.cuda.empty_cache()


def normal(gen, *shape, std=1.0):
    import torch
    return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def generator(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def near(got, ref, tol):
    assert ((got.double() - ref).abs() <= tol).all()


def places(rows, width):
    """Rows around the 2^31st element and at the end."""
    at = 2 ** 31 // width
    assert at + 40 < rows
    return [slice(at - 40, at + 40), slice(rows - 40, rows)]


def test_products_of_many_rows(M):
    import torch
    gen, k = generator(1), 64
    splits = [1000, 262144 + 5000]
    m = sum(splits)
    x, w = normal(gen, m, k), normal(gen, 2, WIDE, k)
    y = M.grouped_gemm_bf16("fprop", splits, x, w)
    for s in places(m, WIDE):
        xd, wd = x[s].double(), w[1].double()
        ref, mag = xd @ wd.t(), xd.abs() @ wd.abs().t()
        near(y[s], ref, (k + 2) * U32 * mag + UBF * ref.abs())
    # and as an operand: its rows reduced over the wide side
    del w
    w = normal(gen, 2, WIDE, k, std=WIDE ** -0.5)
    z = M.grouped_gemm_bf16("dgrad", splits, y, w, out_dtype=torch.float32)
    for s in places(m, WIDE):
        yd, wd = y[s].double(), w[1].double()
        ref, mag = yd @ wd, yd.abs() @ wd.abs()
        near(z[s], ref, (WIDE + 2) * U32 * mag)


def test_weight_gradients_of_many_groups(M):
    import torch
    gen, e = generator(2), 36
    splits = [3] * e
    a, b = normal(gen, 3 * e, WIDE), normal(gen, 3 * e, WIDE)
    dw = M.grouped_gemm_bf16("wgrad", splits, a, b)
    for g in (31, 32, e - 1):
        ad, bd = a[3 * g:3 * g + 3, :80].double(), b[3 * g:3 * g + 3].double()
        ref, mag = ad.t() @ bd, ad.abs().t() @ bd.abs()
        near(dw[g, :80], ref, 5 * U32 * mag + UBF * ref.abs())
    assert torch.equal(dw[e - 1], M.grouped_gemm_bf16("wgrad", [3], a[-3:].contiguous(), b[-3:].contiguous())[0])


def test_gated_rows(M):
    import torch
    gen, k, f = generator(3), 32, WIDE
    m = 2 ** 31 // (2 * f) + 2000
    x, w = normal(gen, m, k), normal(gen, 1, 2 * f, k, std=k ** -0.5)
    pre = torch.empty((m, 2 * f), device="cuda")
    h = M.grouped_gated_fwd("swiglu", [m], x, w, pre=pre)
    for s in places(m, 2 * f):
        xd, wd = x[s].double(), w[0].double()
        ref, mag = xd @ wd.t(), xd.abs() @ wd.abs().t()
        near(pre[s], ref, (k + 2) * U32 * mag)
        v, dg, _, mag_v, mag_g = act64("swiglu", ref[:, :f], ref[:, f:])
        d = (k + 2) * U32 * mag
        # (the derivatives bound the effect of the sums' error, twice them as they change over it)
        tol = 2 * (dg.abs() + mag_g) * d[:, :f] + (ref[:, :f].abs() + 1) * d[:, f:] + UACT * mag_v
        near(h[s], v, tol + UBF * v.abs())
    dy, w2 = normal(gen, m, k), normal(gen, 1, k, f)
    dp = torch.empty(m, device="cuda")
    dpre = M.grouped_gated_bwd("swiglu", [m], dy, w2, pre, dprobs=dp)
    for s in places(m, 2 * f):
        da, mag = dy[s].double() @ w2[0].double(), dy[s].double().abs() @ w2[0].double().abs()
        p = pre[s].double()
        a, dg, du, mag_a, mag_g = act64("swiglu", p[:, :f], p[:, f:])
        d = (k + 2) * U32 * mag
        ref = torch.cat([da * dg, da * du], 1)
        tol = torch.cat([d * dg.abs() + UACT * da.abs() * mag_g, d * du.abs() + UACT * (da * du).abs()], 1)
        near(dpre[s], ref, tol + UBF * ref.abs())
        near(dp[s], (da * a).sum(1), (d * a.abs() + (UACT + (f + 8) * U32) * da.abs() * mag_a).sum(1))


def test_4bit_rows(M):
    import torch
    k, group = 64, 32
    m = 2 ** 31 // WIDE + 3000
    w = weights(1, WIDE, k, group, True, 4)
    x = normal(generator(5), m, k)
    y = M.grouped_gemm_w4([m], x, M.w4_pack(*[t.cuda() for t in w]))
    v, scales = values64(*w)[0].cuda(), w[1][0].double().abs().cuda()
    for s in places(m, WIDE):
        xd = x[s].double()
        ref = xd @ v.t()
        xs = xd.abs().view(xd.shape[0], k // group, group).sum(2)
        tol = (2 * (group + 2) + k // group + 4) * U32 * 31 * (xs @ scales.t())
        near(y[s], ref, tol + (U32 + UBF) * ref.abs())


def test_long_gradient(M):
    import math
    import torch
    n = 2 ** 31 + 70001
    g = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    gen, total = generator(6), []
    for lo in range(0, n, 2 ** 27):
        v = g[lo:lo + 2 ** 27]
        v.copy_(torch.randn(v.numel(), generator=gen, device="cuda"))
        total.append((v.float() ** 2).sum(dtype=torch.float64).item())
    ref = math.sqrt(math.fsum(total))
    ends = [slice(2 ** 31 - 5000, 2 ** 31 + 5000), slice(n - 5000, n)]
    src = [g[s].double() for s in ends]
    norm = M.clip_grad_norm([g], 1.0)
    # (a BF16 value's square is exact in FP32)
    assert abs(norm.item() - ref) <= 1.01 * U32 * ref
    for s, v in zip(ends, src):
        want = v / (ref + 1e-6)
        near(g[s], want, (UBF + 3 * U32) * want.abs())
