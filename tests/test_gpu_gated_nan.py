"""NaN and infinities in a row of the gated kernels: what the activation's formula gives of them, in that row only.

The clamps of the clamped SwiGLU keep a NaN: a value and both derivatives are NaN where gate or up is.  Infinities are
clamped like other values, but for a gate of -inf (-inf times a sigmoid of 0 is NaN, for SwiGLU too).
"""

import math

import pytest

from test_gpu_gated import ALPHA, BETA, KINDS, LIMIT, U32, UACT, UBF, act_of, cuda, gated_case, normal
from test_gpu_w4 import weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_scaled_amd as m
    return m


def formula(kind, g, u):
    """(value, by gate, by up) in 64 bits.  By gate: a NaN of either reaches it; by up: for the clamped kind too."""
    import torch
    if kind == "clamped_swiglu":
        gc = torch.where(g > LIMIT, LIMIT, g)
        uc = torch.where(u > LIMIT, LIMIT, torch.where(u < -LIMIT, -LIMIT, u))
        s = torch.sigmoid(ALPHA * gc)
        nan = torch.isnan(g) | torch.isnan(u)
        by_g = torch.where(g > LIMIT, 0.0, (uc + BETA) * s * (1 + ALPHA * gc * (1 - s)))
        by_u = torch.where(u.abs() > LIMIT, 0.0, gc * s)
        # (a gate of -inf: its silu is NaN, and so is what up's derivative, masked or not, is made of)
        by_u = torch.where(torch.isnan(gc * s), math.nan, by_u)
        return gc * s * (uc + BETA), torch.where(nan, math.nan, by_g), torch.where(nan, math.nan, by_u)
    s = torch.sigmoid(g)
    if kind == "glu":
        return s * u, u * (s * (1 - s)), s
    return g * s * u, u * s * (1 + g * (1 - s)), g * s


def same(got, ref, tol, what):
    """NaN where the reference has it, the same infinities, and the rest within tol."""
    import torch
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), (what, got, ref)
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), what
    ok = ~(inf | torch.isnan(ref))
    assert ((got[ok] - ref[ok]).abs() <= (tol if isinstance(tol, float) else tol[ok])).all(), what


# few rows in both forms, and tiles of 64, 128 and 256
FORWARD = [([3, 0, 14], 72, 136), ([3, 30], 4104, 24), ([70, 0, 129], 72, 136), ([100, 300, 0, 77], 3200, 40), ([1000, 500], 4096 - 8, 24)]


@pytest.mark.parametrize("pre_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("splits,f,k", FORWARD)
@pytest.mark.parametrize("kind", KINDS)
def test_forward(M, kind, splits, f, k, pre_dtype):
    import torch
    x, w, b, p = cuda(*gated_case(kind, splits, f, k, seed=21))
    m = sum(splits)
    bad = {0: math.nan, 2: math.inf, m - 1: -math.inf}
    keep = [i for i in range(m) if i not in bad]
    clean = M.grouped_gated_fwd(act_of(kind), splits, x, w, b, p)
    for i, v in bad.items():
        x[i, 7] = v
    pre = torch.empty((m, 2 * f), dtype=torch.float32 if pre_dtype == "f32" else torch.bfloat16, device="cuda")
    h = M.grouped_gated_fwd(act_of(kind), splits, x, w, b, p, pre=pre)
    assert torch.equal(h[keep], clean[keep]) and not h[keep].isnan().any()
    rows = list(bad)
    got = pre[rows].double().cpu()
    # (a weight of 0 makes NaN of an infinity; the others keep or turn its sign)
    e = [next(g for g in range(len(splits)) if i < sum(splits[:g + 1])) for i in rows]
    want = torch.stack([w[g, :, 7].double().cpu() * v for g, v in zip(e, bad.values())])
    assert torch.equal(got.nan_to_num(0.5), want.nan_to_num(0.5))
    assert got[0].isnan().all()
    ref = formula(kind, got[:, :f], got[:, f:])[0] * p[rows].double().cpu()[:, None]
    assert ref[0].isnan().all()
    # what is finite is clamped: the magnitudes of up + beta, 2, are at most twice its value
    same(h[rows], ref, (UBF + 3 * UACT) * ref.abs().nan_to_num(0.0, 0.0, 0.0), "h")


def special(f, gen):
    """Gates and ups [rows, f]: every pair of NaN, the infinities, values beyond and inside the limit, shuffled."""
    import torch
    v = torch.tensor([math.nan, math.inf, -math.inf, 3.0, -3.0, 0.75, -0.75, 0.0])
    pairs = torch.cartesian_prod(v, v)
    pairs = pairs[torch.randperm(64, generator=gen)].repeat(-(-f // 64) + 1, 1)[:f]
    return pairs[:, 0], pairs[:, 1]


@pytest.mark.parametrize("pre_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("splits,f,n", [([5, 0, 20], 72, 136), ([100, 300, 0, 77], 6400, 24), ([1000, 500], 8192 - 8, 24)])
@pytest.mark.parametrize("kind", KINDS)
def test_backward(M, kind, splits, f, n, pre_dtype):
    import torch
    gen = torch.Generator().manual_seed(22)
    m, e = sum(splits), len(splits)
    dt = torch.float32 if pre_dtype == "f32" else torch.bfloat16
    dy, w2 = normal(gen, m, n), normal(gen, e, n, f, std=n ** -0.5)
    pre = torch.randn(m, 2 * f, generator=gen).to(dt)
    p = torch.rand(m, generator=gen) + 0.5
    rows = [1, m - 1]
    clean = M.grouped_gated_bwd(act_of(kind), splits, *cuda(dy, w2, pre, p))
    for r in rows:
        pre[r, :f], pre[r, f:] = special(f, gen)
    h = torch.empty((m, f), dtype=torch.bfloat16, device="cuda")
    dp = torch.empty(m, device="cuda")
    got = M.grouped_gated_bwd(act_of(kind), splits, *cuda(dy, w2, pre, p), h=h, dprobs=dp)
    keep = [i for i in range(m) if i not in rows]
    assert torch.equal(got[keep], clean[keep]) and dp[keep].isfinite().all() and dp[rows].isnan().all()
    da = torch.stack([dy[r].double() @ w2[g].double() for r, g in zip(rows, (0, e - 1))])
    mag = torch.stack([dy[r].double().abs() @ w2[g].double().abs() for r, g in zip(rows, (0, e - 1))])
    sure = da.abs() > (n + 2) * U32 * mag  # (elsewhere the sign of an infinity is not determined)
    assert sure.double().mean() > 0.99
    a, by_g, by_u = formula(kind, pre[rows, :f].double(), pre[rows, f:].double())
    s = p[rows].double()[:, None]
    # (the magnitudes of a finite value's terms are below 20)
    same(h[rows], a * s, UBF * (a * s).abs().nan_to_num(0.0, 0.0, 0.0) + 20 * UACT, "h")
    for half, by in ((slice(0, f), by_g), (slice(f, None), by_u)):
        ref = da * s * by
        # (the derivatives' terms: up times 1 + alpha |gate|, none above 20 here)
        tol = UBF * ref.abs().nan_to_num(0.0, 0.0, 0.0) + s * ((n + 2) * U32 * mag * by.abs().nan_to_num(0.0, 0.0, 0.0) + 20 * UACT * da.abs())
        same(got[rows][:, half].cpu()[sure], ref[sure], tol[sure], "dpre")


@pytest.mark.parametrize("kind", KINDS)
def test_a_broken_row_reaches_the_gradients(M, kind):
    """A NaN in one row of x: the weights' gradients of its expert and the norm of all gradients are NaN."""
    import torch
    splits, h, f = [9, 20], 64, 72
    x, w1, b1, p = cuda(*gated_case(kind, splits, f, h, seed=23))
    gen = torch.Generator().manual_seed(24)
    w2, dy = cuda(normal(gen, 2, h, f, std=f ** -0.5), normal(gen, 29, h))
    x[3, 5] = math.nan
    mlp = M.GatedMLP(kind, w1, w2, b1, limit=LIMIT, alpha=ALPHA, beta=BETA)
    y = mlp.forward(x, p, splits)
    g = mlp.backward(dy)
    keep = [i for i in range(29) if i != 3]
    assert y[3].isnan().all() and y[keep].isfinite().all()
    assert g["dx1"][3].isnan().all() and g["dprobs"][3].isnan() and g["dx1"][keep].isfinite().all() and g["dprobs"][keep].isfinite().all()
    for k in ("dw1", "dw2", "db1"):
        assert g[k][0].isnan().all() and g[k][1].isfinite().all(), k
    assert M.grad_norm([g["dw1"], g["dw2"]]).isnan()


@pytest.mark.parametrize("splits,f", [([3, 1], 48), ([16, 9], 48), ([32, 20], 48), ([64, 40], 48), ([4, 2], 8208), ([16, 9], 8208), ([30, 20], 8208)])
@pytest.mark.parametrize("kind", KINDS)
def test_w4(M, kind, splits, f):
    """NaN and infinities of a row both make it NaN: the sums of codes and of x, whose difference is taken, are infinite."""
    import torch
    k, m = 160, sum(splits)
    packed = M.w4_pack(*cuda(*weights(2, 2 * f, k, 32, True, seed=25)))
    x = normal(torch.Generator().manual_seed(26), m, k).cuda()
    clean = M.grouped_gated_w4(act_of(kind), splits, x, packed)
    for bad, v in ((0, math.nan), (1, math.inf), (m - 1, -math.inf)):
        z = x.clone()
        z[bad, 37] = v
        h = M.grouped_gated_w4(act_of(kind), splits, z, packed)
        keep = [i for i in range(m) if i != bad]
        assert torch.equal(h[keep], clean[keep]) and h[bad].isnan().all(), (bad, v)


def test_w4_block(M):
    import torch
    e, h, f = 2, 128, 96
    w1, w2 = M.w4_pack(*cuda(*weights(e, 2 * f, h, 32, True, 27))), M.w4_pack(*cuda(*weights(e, h, f, 32, False, 28)))
    x = normal(torch.Generator().manual_seed(29), 12, h).cuda()
    x[4, 1] = math.nan
    y = M.W4GatedMLP("clamped_swiglu", w1, w2).forward(x, None, [5, 7])
    assert y[4].isnan().all() and y[[i for i in range(12) if i != 4]].isfinite().all()
