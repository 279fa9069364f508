"""Every form of the few-rows MXFP4 product (gemm_mxfp4_rows_kernel<MT, NT, D>: tiles of 16 MT x 16 NT, D units in a
wave's ring) against 64-bit products of the decoded operands, in every mode and output type, with K remainders and
device-resident split sizes.  `rows_variant` restates the library's choice, so that the cases can be seen to reach
each form."""

import pytest

from test_gpu_mxfp4_large import N, _close, _colwise, _rowwise  # noqa: F401 (N: fixture)

FORMS = {(1, 2, 1), (1, 2, 2), (4, 4, 1), (2, 4, 1), (2, 2, 1), (2, 2, 2)}


def rows_variant(mode, splits, m, n, cap=None):
    """(MT, NT, D) of a launch, or None for the 256 x 256 tiles; `cap`: the row capacity of device-resident splits."""
    up = lambda a, b: -(-a // b)
    e = len(splits)

    def tiles(tm, tn):
        if mode == "wgrad":
            rows = up(m, tm) * e
        elif cap is not None:
            rows = up(cap, tm) + e
        else:
            rows = sum(up(s, tm) for s in splits)
        return rows * up(n, tn)

    if mode == "wgrad":
        most = m
    elif cap is not None:
        most = min(cap, max(16, 2 * cap // e))
    else:
        most = max(splits)
    if most > 64 and tiles(64, 64) > 1024:
        return None
    if most <= 16:
        return (1, 2, 1) if tiles(16, 32) >= 512 else (1, 2, 2)
    if most > 32 and tiles(64, 64) >= 512:
        return (4, 4, 1)
    if tiles(32, 64) >= 512:
        return (2, 4, 1)
    return (2, 2, 1) if tiles(32, 32) >= 512 else (2, 2, 2)


# rows of the groups, n, capacity of device-resident splits or None, form
PRODUCTS = [
    ([2, 0, 16, 1] * 4, 4128, None, (1, 2, 1)),
    ([2, 0, 5, 1] * 4, 4128, 40, (1, 2, 1)),
    ([16, 0, 3], 288, None, (1, 2, 2)),
    ([40, 0, 0, 0] * 4, 288, 160, (2, 2, 2)),           # a group past what the capacity lets expect
    ([64, 33, 0, 50] * 4, 4128, None, (4, 4, 1)),
    ([100, 0, 0, 23] * 4, 4128, 500, (4, 4, 1)),
    ([32, 17, 0, 5] * 4, 4128, None, (2, 4, 1)),
    ([90, 0, 1, 5] * 2, 4128, 200, (4, 4, 1)),
    ([30, 0, 90, 5] * 2, 2080, 128 * 2, (2, 4, 1)),
    ([32, 17, 0, 5] * 4, 1376, None, (2, 2, 1)),
    ([50, 0, 1, 9] * 4, 800, 250, (2, 2, 1)),
    ([33, 64, 65], 288, None, (2, 2, 2)),
]
# rows of the groups, m, n, form
GRADIENTS = [
    ([300, 0, 1, 129] * 2, 64, 4128, (4, 4, 1)),
    ([37, 0, 257, 128], 96, 4128, (4, 4, 1)),
    ([300, 0, 1, 129] * 2, 32, 4128, (2, 4, 1)),
    ([130, 0, 5] * 4, 32, 1376, (2, 2, 1)),
    ([130, 0, 5], 32, 160, (2, 2, 2)),
]


def test_cases_reach_every_form():
    for splits, n, cap, form in PRODUCTS:
        assert rows_variant("fprop", splits, None, n, cap) == form, (splits, n, cap)
        assert cap is None or sum(splits) <= cap
    for splits, m, n, form in GRADIENTS:
        assert rows_variant("wgrad", splits, m, n) == form, (splits, m, n)
    assert {p[-1] for p in PRODUCTS} == FORMS and {p[-1] for p in PRODUCTS if p[2]} >= {(1, 2, 1), (4, 4, 1), (2, 4, 1), (2, 2, 1), (2, 2, 2)}


@pytest.mark.gpu
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("mode,k", [("fprop", 32), ("fprop", 288), ("fprop", 1120), ("fprop", 2304), ("dgrad", 160), ("dgrad", 1056)])
@pytest.mark.parametrize("splits,n,cap,form", PRODUCTS, ids=lambda v: str(v))
def test_products(N, splits, n, cap, form, mode, k, out, bias):  # noqa: F811
    import torch
    gen = torch.Generator(device="cuda").manual_seed(k + n)
    e, m = len(splits), sum(splits)
    dg, rows = None, m
    if cap:
        rows = cap
        dg = N.DeviceGroups(e, cap)
        dg.splits.copy_(torch.tensor(splits))
        dg.update()
    a, a64 = _rowwise(N, gen, splits, k, dg)
    if mode == "fprop":
        b, b64 = _rowwise(N, gen, [n] * e, k)
        b64 = b64.view(e, n, k)
    else:
        b, b64 = _colwise(N, gen, [k] * e, n)
    bv = torch.randn((e, n), generator=gen, device="cuda", dtype=torch.bfloat16)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    full = torch.full((rows + 64, n), 7.0, dtype=dt, device="cuda")
    c = full[32:32 + rows]
    print("case:", splits, n, cap, form, mode, k, out, bias, flush=True)
    N.grouped_gemm_mx(mode, "mxfp4", dg or splits, rows, n, k, a, b, c, bias=bv if bias else None)
    torch.cuda.synchronize()
    assert bool((full[:32] == 7.0).all()) and bool((c[m:] == 7.0).all()) and bool((full[32 + rows:] == 7.0).all())
    lo = 0
    for g, r in enumerate(splits):
        x, w = a64[lo:lo + r], b64[g].t().contiguous()
        ref, size = x @ w, x.abs() @ w.abs()
        if bias:
            ref, size = ref + bv[g].double(), size + bv[g].double().abs()
        _close(c[lo:lo + r], ref, size, k)
        lo += r


@pytest.mark.gpu
@pytest.mark.parametrize("device_splits", [False, True])
@pytest.mark.parametrize("out,accumulate", [("f32", False), ("f32", True), ("bf16", False)])
@pytest.mark.parametrize("splits,m,n,form", GRADIENTS, ids=lambda v: str(v))
def test_weight_gradients(N, splits, m, n, form, out, accumulate, device_splits):  # noqa: F811
    import torch
    gen = torch.Generator(device="cuda").manual_seed(n + m)
    e, k = len(splits), sum(splits)
    dg, cap = None, k
    if device_splits:
        cap = k + 200
        dg = N.DeviceGroups(e, cap)
        dg.splits.copy_(torch.tensor(splits))
        dg.update()
    a, a64 = _colwise(N, gen, splits, m, dg)
    b, b64 = _colwise(N, gen, splits, n, dg)
    full = torch.randn((e + 2, m, n), generator=gen, device="cuda").to(torch.float32 if out == "f32" else torch.bfloat16)
    old = full.clone()
    c = full[1:1 + e]
    print("case:", splits, m, n, form, out, accumulate, device_splits, flush=True)
    N.grouped_gemm_mx("wgrad", "mxfp4", dg or splits, m, n, cap, a, b, c, accumulate=accumulate)
    torch.cuda.synchronize()
    assert torch.equal(full[0], old[0]) and torch.equal(full[-1], old[-1])
    for g, r in enumerate(splits):
        bt = b64[g].t().contiguous()
        ref, size = a64[g] @ bt, a64[g].abs() @ bt.abs()
        if accumulate:
            ref, size = ref + old[1 + g].double(), size + old[1 + g].double().abs()
        _close(c[g], ref, size, r + 128)


@pytest.mark.gpu
@pytest.mark.parametrize("splits,n,cap,form", [p for p in PRODUCTS if not p[2]], ids=lambda v: str(v))
def test_repeated_launches_are_bitwise_equal(N, splits, n, cap, form):  # noqa: F811
    import torch
    gen = torch.Generator(device="cuda").manual_seed(0)
    m, k = sum(splits), 1120
    a, _ = _rowwise(N, gen, splits, k)
    b, _ = _rowwise(N, gen, [n] * len(splits), k)
    c = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    N.grouped_gemm_mx("fprop", "mxfp4", splits, m, n, k, a, b, c)
    for _ in range(10):
        d = torch.full_like(c, float("nan"))
        N.grouped_gemm_mx("fprop", "mxfp4", splits, m, n, k, a, b, d)
        assert torch.equal(c, d)
