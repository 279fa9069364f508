"""MXFP4 products large enough for the 256 x 256 tiles, against 64-bit products of the decoded operands: ragged
groups, widths that end inside a tile, one to several whole and partial K steps, every output form."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def N():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from moe_grouped_scaled_amd import _native
    return _native


def _decode(codes, scales):
    """Codes [R, W / 2] and E8M0 codes [R, W / 32] -> 64-bit values [R, W]."""
    import torch
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    lut = torch.cat([mag, -mag])
    v = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], dim=2).reshape(codes.shape[0], -1)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)


def _codes(gen, rows, width):
    import torch
    c = torch.randint(0, 256, (rows, width // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s = torch.randint(118, 126, (rows, width // 32), generator=gen, device="cuda", dtype=torch.uint8)
    return c, s


def _kstep(s):
    """E8M0 codes [R, W / 32] in the K-step grouped layout [steps, R, 4], unused bytes zero."""
    import torch
    r, b = s.shape
    p = torch.zeros((r, -(-b // 4) * 4), dtype=torch.uint8, device="cuda")
    p[:, :b] = s
    return p.view(r, -1, 4).permute(1, 0, 2).contiguous()


def _rowwise(N, gen, splits, width, dg=None):
    """A rowwise tensor of random codes and its 64-bit values; with device-resident splits every byte past the rows in
    use is 0xFF (no number)."""
    m = sum(splits)
    c, s = _codes(gen, m, width)
    t = N.QTensor("mxfp4", False, dg or splits, width)
    t.data.fill_(0xFF)
    t.scales.fill_(0xFF)
    t.data[:c.numel()] = c.view(-1)
    t.scales.view(-(-width // 128), -1, 4)[:, :m] = _kstep(s)
    return t, _decode(c, s)


def _colwise(N, gen, splits, width, dg=None):
    """A columnwise tensor of random codes (padding tokens zero) and, per group, its 64-bit values [width, m_g]."""
    import torch
    t = N.QTensor("mxfp4", True, dg or splits, width)
    t.data.fill_(0xFF)
    t.scales.fill_(0xFF)
    vals, at = [], 0
    for m in splits:
        mp = -(-m // 128) * 128
        c, s = _codes(gen, width, mp)
        c[:, (m + 1) // 2:] = 0
        if m % 2:
            c[:, m // 2] &= 15
        s[:, -(-m // 32):] = 0
        t.data[width * at // 2:width * (at + mp) // 2] = c.view(-1)
        t.scales[width * at // 32:width * (at + mp) // 32] = _kstep(s).view(-1)
        vals.append(_decode(c, s)[:, :m] if m else torch.zeros((width, 0), dtype=torch.float64, device="cuda"))
        at += mp
    return t, vals


def _close(got, ref, size, k):
    # one rounding of FP32 per block of 32 products (exact among themselves) and a few in the epilogue; BF16: one more
    import torch
    tol = (k / 32 + 8) * 2.0 ** -23 * size
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    assert bool(((got.double() - ref).abs() <= tol).all())


SPLITS = [700, 0, 65, 300]


@pytest.mark.parametrize("device_splits", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("mode,k", [("fprop", 32), ("fprop", 256), ("fprop", 288), ("fprop", 512), ("fprop", 800), ("fprop", 1120),
                                    ("dgrad", 544), ("dgrad", 768)])
def test_products(N, mode, k, out, bias, device_splits):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(k)
    e, m, n = len(SPLITS), sum(SPLITS), 4128
    dg, cap = None, m
    if device_splits:
        cap = m + 100
        dg = N.DeviceGroups(e, cap)
        dg.splits.copy_(torch.tensor(SPLITS))
        dg.update()
    a, a64 = _rowwise(N, gen, SPLITS, k, dg)
    if mode == "fprop":
        b, b64 = _rowwise(N, gen, [n] * e, k)
        b64 = b64.view(e, n, k)
    else:
        b, b64 = _colwise(N, gen, [k] * e, n)
    bv = torch.randn((e, n), generator=gen, device="cuda", dtype=torch.bfloat16)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    full = torch.full((cap + 64, n), 7.0, dtype=dt, device="cuda")
    c = full[32:32 + cap]
    print("case:", mode, k, out, bias, device_splits, flush=True)
    N.grouped_gemm_mx(mode, "mxfp4", dg or SPLITS, cap, n, k, a, b, c, bias=bv if bias else None)
    torch.cuda.synchronize()
    assert bool((full[:32] == 7.0).all()) and bool((c[m:] == 7.0).all()) and bool((full[32 + cap:] == 7.0).all())
    lo = 0
    for g, rows in enumerate(SPLITS):
        x, w = a64[lo:lo + rows], b64[g]
        ref, size = x @ w.t().contiguous(), x.abs() @ w.t().contiguous().abs()
        if bias:
            ref, size = ref + bv[g].double(), size + bv[g].double().abs()
        _close(c[lo:lo + rows], ref, size, k)
        lo += rows


@pytest.mark.parametrize("device_splits", [False, True])
@pytest.mark.parametrize("out,accumulate", [("f32", False), ("f32", True), ("bf16", False)])
@pytest.mark.parametrize("splits", [[300, 0, 513], [1, 129, 256], [1000]], ids=str)
def test_weight_gradients(N, splits, out, accumulate, device_splits):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(len(splits))
    e, m, mw, n = len(splits), sum(splits), 2080, 2144
    dg, cap = None, m
    if device_splits:
        cap = m + 200
        dg = N.DeviceGroups(e, cap)
        dg.splits.copy_(torch.tensor(splits))
        dg.update()
    a, a64 = _colwise(N, gen, splits, mw, dg)
    b, b64 = _colwise(N, gen, splits, n, dg)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    full = torch.randn((e + 2, mw, n), generator=gen, device="cuda").to(dt)
    old = full.clone()
    c = full[1:1 + e]
    print("case:", splits, out, accumulate, device_splits, flush=True)
    N.grouped_gemm_mx("wgrad", "mxfp4", dg or splits, mw, n, cap, a, b, c, accumulate=accumulate)
    torch.cuda.synchronize()
    assert torch.equal(full[0], old[0]) and torch.equal(full[-1], old[-1])
    for g, rows in enumerate(splits):
        bt = b64[g].t().contiguous()
        ref, size = a64[g] @ bt, a64[g].abs() @ bt.abs()
        if accumulate:
            ref, size = ref + old[1 + g].double(), size + old[1 + g].double().abs()
        _close(c[g], ref, size, rows + 128)


def test_repeated_launches_are_bitwise_equal(N):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(0)
    a, _ = _rowwise(N, gen, [2000, 500, 1500], 1120)
    b, _ = _rowwise(N, gen, [4128] * 3, 1120)
    c = torch.empty((4000, 4128), dtype=torch.bfloat16, device="cuda")
    N.grouped_gemm_mx("fprop", "mxfp4", [2000, 500, 1500], 4000, 4128, 1120, a, b, c)
    for _ in range(20):
        d = torch.full_like(c, float("nan"))
        N.grouped_gemm_mx("fprop", "mxfp4", [2000, 500, 1500], 4000, 4128, 1120, a, b, d)
        assert torch.equal(c, d)
