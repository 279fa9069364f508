"""The grouped BF16 products and the gated block's kernels against their formulas in 64 bits.

Bounds, element by element: a sum of k products of BF16 numbers in FP32 (any order) is off by at most
k 2^-24 sum |a b|; rounding to BF16 adds 2^-8 of the value; the activation's own arithmetic (an exponential and a
reciprocal of about 2^-22 each, a few roundings) at most 2^-19 of the sum of the magnitudes it adds up.
"""

import math

import pytest

pytestmark = pytest.mark.gpu

KINDS = ("swiglu", "clamped_swiglu", "glu")
LIMIT, ALPHA, BETA = 1.5, 1.25, 0.5
U32, UBF, UACT = 2.0 ** -24, 2.0 ** -8, 2.0 ** -19


@pytest.fixture(scope="module")
def M():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_scaled_amd as m
    return m


def act_of(kind):
    from moe_grouped_scaled_amd import act_params
    return act_params(kind, limit=LIMIT, alpha=ALPHA, beta=BETA)


def normal(gen, *shape, std=1.0):
    import torch
    return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16)


def act64(kind, g, u):
    """(value, by gate, by up, sum of the magnitudes of the value's and the derivatives' terms)"""
    import torch
    if kind == "clamped_swiglu":
        gc, uc = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
        s = torch.sigmoid(ALPHA * gc)
        a = gc * s * (uc + BETA)
        dg = torch.where(g <= LIMIT, (uc + BETA) * s * (1 + ALPHA * gc * (1 - s)), 0.0)
        du = torch.where(u.abs() <= LIMIT, gc * s, 0.0)
        mag_g = (uc.abs() + BETA) * s * (1 + ALPHA * gc.abs())
        return a, dg, du, (gc * s).abs() * (uc.abs() + BETA), mag_g
    s = torch.sigmoid(g)
    if kind == "glu":
        return s * u, s * (1 - s) * u, s, (s * u).abs(), s * u.abs()
    return g * s * u, u * s * (1 + g * (1 - s)), g * s, (g * s * u).abs(), (u * s).abs() * (1 + g.abs())


def check(got, ref, tol, what):
    import torch
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = (got - ref).abs() > tol + 1e-30
    bad |= ~torch.isfinite(got)
    assert not bad.any(), "%s: %d of %d outside, first %s: %r instead of %r, allowed %r" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), got[bad][0].item(), ref[bad][0].item(),
        (tol if isinstance(tol, float) else tol[bad][0].item()))


def bounds(splits):
    lo = 0
    for g, m in enumerate(splits):
        yield g, slice(lo, lo + m)
        lo += m


SPLITS = {
    "one_row": [1],
    "few": [3, 0, 1, 16, 17, 0, 31],
    "ragged": [70, 0, 129, 1, 64],
    "empty": [0, 0],
}


def product64(mode, splits, a, b, bias=None):
    """(C, sum of magnitudes) in 64 bits"""
    import torch
    a, b = a.double(), b.double()
    if mode == "wgrad":
        c = torch.zeros((len(splits), a.shape[1], b.shape[1]), dtype=torch.float64)
        mag = torch.zeros_like(c)
        for g, at in bounds(splits):
            c[g], mag[g] = a[at].t() @ b[at], a[at].abs().t() @ b[at].abs()
        return c, mag
    n = b.shape[1] if mode == "fprop" else b.shape[2]
    c = torch.zeros((a.shape[0], n), dtype=torch.float64)
    mag = torch.zeros_like(c)
    for g, at in bounds(splits):
        w = b[g].t() if mode == "fprop" else b[g]
        c[at], mag[at] = a[at] @ w, a[at].abs() @ w.abs()
        if bias is not None:
            c[at] += bias[g].double()
            mag[at] += bias[g].double().abs()
    return c, mag


def operands(mode, splits, n, k, seed):
    import torch
    gen = torch.Generator().manual_seed(seed)
    m, e = sum(splits), len(splits)
    if mode == "wgrad":
        return normal(gen, m, k), normal(gen, m, n)
    return normal(gen, m, k), normal(gen, *((e, n, k) if mode == "fprop" else (e, k, n)))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(8, 8), (72, 136), (264, 200), (128, 64)])
@pytest.mark.parametrize("split", sorted(SPLITS))
@pytest.mark.parametrize("mode", ["fprop", "dgrad", "wgrad"])
def test_products(M, mode, split, n, k, out):
    import torch
    splits = SPLITS[split]
    a, b = operands(mode, splits, n, k, seed=n + k)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    bias = None
    if mode != "wgrad":
        bias = normal(torch.Generator().manual_seed(1), len(splits), n)
    ref, mag = product64(mode, splits, a, b, bias)
    got = M.grouped_gemm_bf16(mode, splits, a.cuda(), b.cuda(), bias=None if bias is None else bias.cuda(), out_dtype=dt)
    length = max(sum(splits), 1) if mode == "wgrad" else k
    tol = (length + 2) * U32 * mag + (UBF if out == "bf16" else U32) * ref.abs()
    check(got, ref, tol, "c")


# sizes that reach the larger tiles: 128 x 128 and 256 x 256 (by the number of tiles they give)
LARGE = [("fprop", [100, 300, 0, 77], 6400, 40), ("dgrad", [100, 300, 0, 77], 6400, 40), ("wgrad", [40, 0, 9] * 5, 520, 456),
         ("fprop", [1000, 500], 8192 - 8, 200), ("dgrad", [1000, 500], 8192 - 8, 200), ("wgrad", [70, 0, 129] * 4, 1032, 1000)]
# groups whose last tile has at most half of its rows, of both sizes
HALVES = [[1000, 300, 20, 0, 500, 1, 384], [130, 50, 0, 192, 1]]
LARGE += [(mode, splits, n, k) for mode in ("fprop", "dgrad") for splits, n, k in zip(HALVES, (8192 - 8, 6400), (200, 136))]


@pytest.mark.parametrize("mode,splits,n,k", LARGE)
def test_products_on_larger_tiles(M, mode, splits, n, k):
    import torch
    a, b = operands(mode, splits, n, k, seed=5)
    ref, mag = product64(mode, splits, a, b)
    length = max(splits) if mode == "wgrad" else k
    for dt, u in ((torch.bfloat16, UBF), (torch.float32, U32)):
        got = M.grouped_gemm_bf16(mode, splits, a.cuda(), b.cuda(), out_dtype=dt)
        check(got, ref, (length + 2) * U32 * mag + u * ref.abs(), "c")


@pytest.mark.parametrize("mode", ["fprop", "dgrad", "wgrad"])
def test_accumulate(M, mode):
    import torch
    splits, n, k = [5, 0, 40], 72, 88
    a, b = operands(mode, splits, n, k, seed=2)
    ref, mag = product64(mode, splits, a, b)
    c = torch.randn(ref.shape, generator=torch.Generator().manual_seed(3))
    got = M.grouped_gemm_bf16(mode, splits, a.cuda(), b.cuda(), c.cuda(), accumulate=True)
    check(got, ref + c.double(), (90 * U32) * mag + U32 * (ref.abs() + c.double().abs()), "c")


@pytest.mark.parametrize("mode", ["fprop", "dgrad", "wgrad"])
@pytest.mark.parametrize("n,k,splits", [(40, 72, [3, 20, 50]), (264, 200, [70, 20, 129])])
def test_other_groups_do_not_reach_a_group(M, mode, n, k, splits):
    """NaN and infinities in the rows and weights of the other experts, and behind the tensors' ends."""
    import torch
    a, b = operands(mode, splits, n, k, seed=4)
    ref, _ = product64(mode, splits, a, b)
    clean = M.grouped_gemm_bf16(mode, splits, a.cuda(), b.cuda())
    lo, hi = splits[0], splits[0] + splits[1]
    for keep, at in ((0, slice(0, lo)), (1, slice(lo, hi)), (2, slice(hi, None))):
        pa = torch.full_like(a, math.nan)
        pa[at] = a[at]
        pb = torch.full_like(b, math.inf)
        if mode == "wgrad":
            pb[at] = b[at]
        else:
            pb[keep] = b[keep]
        big_a = torch.full((a.shape[0] + 64, a.shape[1]), math.nan, dtype=torch.bfloat16, device="cuda")
        big_a[:a.shape[0]] = pa.cuda()
        got = M.grouped_gemm_bf16(mode, splits, big_a[:a.shape[0]], pb.cuda())
        sel = keep if mode == "wgrad" else at
        assert torch.equal(got[sel], clean[sel])


def check_pre(out, pre, dpre, kind, f):
    """[gate | up]: in FP32 the sums themselves; in BF16 to nearest, or for the clamped kind to the same side of the clamps.  Then a value within half a
    step of a limit moves by up to the whole step to the first one on its side, 2 x 2^-8 of it.  Sides are compared
    where the sum's own error does not reach the limit."""
    import torch
    if out.dtype == torch.float32:
        check(out, pre, dpre, "pre")
        return
    u = torch.full_like(pre, UBF)
    if kind == "clamped_swiglu":
        d = (pre.abs() - LIMIT).abs()
        u[d <= UBF * LIMIT * 1.01] = 2 * UBF
        got = out.detach().double().cpu()
        sure = d > dpre
        beyond = lambda v: torch.cat([v[:, :f] > LIMIT, v[:, f:].abs() > LIMIT], 1)
        assert torch.equal(beyond(got)[sure], beyond(pre)[sure])
    check(out, pre, dpre + u * pre.abs(), "pre")


def gated_case(kind, splits, f, k, seed, bias=True, probs=True):
    import torch
    gen = torch.Generator().manual_seed(seed)
    m, e = sum(splits), len(splits)
    x, w = normal(gen, m, k), normal(gen, e, 2 * f, k, std=k ** -0.5)
    b = normal(gen, e, 2 * f, std=0.5) if bias else None
    p = torch.rand(m, generator=gen) if probs else None
    return x, w, b, p


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def gated64(kind, splits, x, w, b, p):
    """h and pre with their bounds before rounding."""
    import torch
    f = w.shape[1] // 2
    pre, mag = product64("fprop", splits, x, w, b)
    d = (x.shape[1] + 2) * U32 * mag
    a, dg, du, mag_a, mag_g = act64(kind, pre[:, :f], pre[:, f:])
    s = torch.ones(x.shape[0], 1, dtype=torch.float64) if p is None else p.double()[:, None]
    # the derivatives bound the effect of the sums' error (twice them: they change a little over it; at the clamp
    # the other side's derivative counts)
    slope_u = mag_a.new_tensor(1.0) * (pre[:, :f].clamp(max=LIMIT if kind == "clamped_swiglu" else math.inf).abs() + 1)
    tol = s * (2 * (dg.abs() + mag_g) * d[:, :f] + slope_u * d[:, f:] + UACT * mag_a)
    return a * s, tol, pre, d


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("f,k", [(8, 8), (72, 136), (264, 200)])
@pytest.mark.parametrize("split", sorted(SPLITS))
def test_gated_forward(M, kind, split, f, k):
    import torch
    splits = SPLITS[split]
    for bias, probs in ((True, True), (False, False)):
        x, w, b, p = gated_case(kind, splits, f, k, seed=f, bias=bias, probs=probs)
        ref, tol, pre, dpre = gated64(kind, splits, x, w, b, p)
        xg, wg, bg, pg = cuda(x, w, b, p)
        for dt in (torch.bfloat16, torch.float32):
            out = torch.full((sum(splits), 2 * f), math.nan, dtype=dt, device="cuda")
            h = M.grouped_gated_fwd(act_of(kind), splits, xg, wg, bg, pg, pre=out)
            check(h, ref, tol + UBF * ref.abs(), "h")
            check_pre(out, pre, dpre, kind, f)
        assert torch.equal(h, M.grouped_gated_fwd(act_of(kind), splits, xg, wg, bg, pg))


@pytest.mark.parametrize("splits,f,k", [([100, 300, 0, 77], 3200, 40), ([1000, 500], 4096 - 8, 200), (HALVES[0], 4096 - 8, 200), (HALVES[1], 3200, 136)])
def test_gated_forward_on_larger_tiles(M, splits, f, k):
    import torch
    x, w, b, p = gated_case("swiglu", splits, f, k, seed=7)
    ref, tol, pre, dpre = gated64("swiglu", splits, x, w, b, p)
    xg, wg, bg, pg = cuda(x, w, b, p)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.empty((sum(splits), 2 * f), dtype=dt, device="cuda")
        h = M.grouped_gated_fwd(act_of("swiglu"), splits, xg, wg, bg, pg, pre=out)
        check(h, ref, tol + UBF * ref.abs(), "h")
        check_pre(out, pre, dpre, "swiglu", f)


def check_backward(M, kind, splits, f, n, seed, probs, pre_dtype):
    import torch
    gen = torch.Generator().manual_seed(seed)
    m, e = sum(splits), len(splits)
    dy, w2 = normal(gen, m, n), normal(gen, e, n, f, std=n ** -0.5)
    pre = (torch.randn(m, 2 * f, generator=gen) * 1.5).to(pre_dtype)
    p = torch.rand(m, generator=gen) if probs else None
    da, mag = product64("dgrad", splits, dy, w2)
    d = (n + 2) * U32 * mag
    a, dg, du, mag_a, mag_g = act64(kind, pre[:, :f].double(), pre[:, f:].double())
    s = torch.ones(m, 1, dtype=torch.float64) if p is None else p.double()[:, None]
    ref = torch.cat([da * s * dg, da * s * du], dim=1)
    tol = torch.cat([s * (d * dg.abs() + UACT * da.abs() * mag_g), s * (d * du.abs() + UACT * (da * du).abs())], dim=1)
    h = torch.full((m, f), math.nan, dtype=torch.bfloat16, device="cuda")
    dp = torch.full((m,), math.nan, device="cuda")
    dyg, w2g, preg, pg = cuda(dy, w2, pre, p)
    got = M.grouped_gated_bwd(act_of(kind), splits, dyg, w2g, preg, pg, h=h, dprobs=dp)
    check(got, ref, tol + UBF * ref.abs(), "dpre")
    check(h, a * s, UACT * mag_a + UBF * (a * s).abs(), "h")
    check(dp, (da * a).sum(1), (d * a.abs() + (UACT + (f + 8) * U32) * da.abs() * mag_a).sum(1), "dprobs")
    # nothing that is asked for changes the rest
    assert torch.equal(got, M.grouped_gated_bwd(act_of(kind), splits, dyg, w2g, preg, pg))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("f,n", [(8, 8), (72, 136), (264, 200)])
@pytest.mark.parametrize("split", sorted(SPLITS))
def test_gated_backward(M, kind, split, f, n):
    import torch
    for probs, dt in ((True, torch.bfloat16), (True, torch.float32), (False, torch.float32)):
        check_backward(M, kind, SPLITS[split], f, n, seed=n, probs=probs, pre_dtype=dt)


@pytest.mark.parametrize("splits,f,n", [([100, 300, 0, 77], 6400, 40), ([1000, 500], 8192 - 8, 200), (HALVES[0], 8192 - 8, 200), (HALVES[1], 6400, 136)])
def test_gated_backward_on_larger_tiles(M, splits, f, n):
    import torch
    for dt in (torch.bfloat16, torch.float32):
        check_backward(M, "swiglu", splits, f, n, seed=9, probs=True, pre_dtype=dt)


@pytest.mark.parametrize("kind", KINDS)
def test_far_gates(M, kind):
    """Gates far from zero: the sigmoid's ends, where exp overflows, and infinities that the definition gives."""
    import torch
    g = torch.tensor([-3e4, -200.0, -89.0, -30.0, 0.0, 30.0, 89.0, 200.0, 3e4, 1.5, -1.5, 2.0]).repeat(2)
    u = torch.tensor([1.0] * 12 + [-2.0] * 12)
    f = g.numel()
    x = torch.zeros(1, 8, dtype=torch.bfloat16)
    w = torch.zeros(1, 2 * f, 8, dtype=torch.bfloat16)
    b = torch.cat([g, u]).to(torch.bfloat16)[None]
    ref, _, _, mag, _ = act64(kind, b[:, :f].double(), b[:, f:].double())
    h = M.grouped_gated_fwd(act_of(kind), [1], *cuda(x, w, b))
    check(h, ref, UBF * ref.abs() + UACT * mag + 1e-38, "h")


def device_groups(splits, cap):
    import torch
    from moe_grouped_scaled_amd import _native as N
    g = N.DeviceGroups(len(splits), cap)
    g.splits.copy_(torch.tensor(splits))
    g.update()
    return g


@pytest.mark.parametrize("splits,cap", [([3, 0, 20], 40), ([100, 0, 300, 7], 500), ([0, 0], 8), ([60, 0, 0, 2], 62)])
@pytest.mark.parametrize("f,k", [(72, 136), (520, 64)])
def test_device_resident_split_sizes(M, splits, cap, f, k):
    """Equal to host split sizes bit for bit; rows past the last used one are neither read nor written."""
    import torch
    m = sum(splits)
    x, w, b, p = cuda(*gated_case("swiglu", splits, f, k, seed=11))
    dg = device_groups(splits, cap)
    wide = lambda t: torch.cat([t, torch.full((cap - m, *t.shape[1:]), math.nan, dtype=t.dtype, device="cuda")])
    mark = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda")
    pre, h = mark(cap, 2 * f), mark(cap, f)
    M.grouped_gated_fwd("swiglu", dg, wide(x), w, b, wide(p), h=h, pre=pre)
    pre0 = mark(m, 2 * f)
    h0 = M.grouped_gated_fwd("swiglu", splits, x, w, b, p, pre=pre0)
    assert (h[m:] == 7).all() and (pre[m:] == 7).all()
    near = lambda got, ref: torch.allclose(got.float(), ref.float(), rtol=2 * UBF, atol=1e-4)
    # (another tile may be picked for the capacity: sums in another order)
    assert near(h[:m], h0) and near(pre[:m], pre0)
    n = 64
    gen = torch.Generator().manual_seed(12)
    dy, w2 = cuda(normal(gen, m, n), normal(gen, len(splits), n, f))
    out, dp = mark(cap, 2 * f), torch.full((cap,), 7.0, device="cuda")
    M.grouped_gated_bwd("swiglu", dg, wide(dy), w2, wide(pre0), wide(p), dpre=out, dprobs=dp)
    dp0 = torch.empty(m, device="cuda")
    out0 = M.grouped_gated_bwd("swiglu", splits, dy, w2, pre0, p, dprobs=dp0)
    assert (out[m:] == 7).all() and (dp[m:] == 7).all()
    assert torch.allclose(out[:m].float(), out0.float(), rtol=2 * UBF, atol=1e-3)
    assert torch.allclose(dp[:m], dp0, rtol=1e-4, atol=1e-2)
    dw = M.grouped_gemm_bf16("wgrad", dg, wide(dy), wide(h0), out_dtype=torch.float32)
    dw0 = M.grouped_gemm_bf16("wgrad", splits, dy, h0, out_dtype=torch.float32)
    assert torch.equal(dw, dw0)
    y = mark(cap, k)
    M.grouped_gemm_bf16("dgrad", dg, wide(pre0), w, y)
    assert (y[m:] == 7).all()


def test_skewed_wgrad_deals_groups(M):
    """One group with most of the rows: the groups are dealt over the XCDs, on host and device split sizes."""
    import torch
    splits = [5, 900, 0, 30, 1, 0, 0, 64]
    a, b = operands("wgrad", splits, 328, 392, seed=13)
    ref, mag = product64("wgrad", splits, a, b)
    ag, bg = cuda(a, b)
    got = M.grouped_gemm_bf16("wgrad", splits, ag, bg, out_dtype=torch.float32)
    check(got, ref, 902 * U32 * mag, "c")
    assert sum(splits) == 1000
    assert torch.equal(got, M.grouped_gemm_bf16("wgrad", device_groups(splits, 1000), ag, bg, out_dtype=torch.float32))
