"""Norm and clipping of many gradients against 64 bits.

Bounds: the sum of squares is FP64 (relative 2^-40 for any order of these sizes), so the norm is its FP32 rounding;
the factor is one rounding to FP32, the product another, the output's own a third: 2 x 2^-24, and 2^-8 where it is BF16.
"""

import math

import pytest

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def M():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_scaled_amd as m
    return m


def make(sizes, seed, std=1.0):
    import torch
    gen = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n, generator=gen) * std
        out.append(t.to(torch.bfloat16 if i % 2 else torch.float32))
    return out


def norm64(ts):
    return math.sqrt(math.fsum((t.double() ** 2).sum().item() for t in ts))


def check(got, src, scale, out_dtype):
    import torch
    ref = src.double().cpu() * scale
    u = 2.0 ** -8 if out_dtype == torch.bfloat16 else 0.0
    tol = (u + 3 * 2.0 ** -24) * ref.abs() + 1e-44  # (subnormal outputs: half a step)
    assert got.dtype == out_dtype
    assert ((got.double().cpu() - ref).abs() <= tol).all()


# (more than 120 tensors: their entries go through the workspace; more than 1024 chunks: a launch of its own adds them)
SIZES = [[1], [7], [2048 * 1100 + 5], [3000000, 70000] + [5] * 200, [65536], [65537, 3, 0, 131072], [1, 2, 3, 4, 5, 1000, 4097], [33] * 300, [200000, 1, 0, 0, 8191, 16]]


@pytest.mark.parametrize("sizes", SIZES)
def test_norm_and_clip(M, sizes):
    import torch
    host = make(sizes, len(sizes))
    ref = norm64(host)
    dev = [t.cuda() for t in host]
    n = M.grad_norm(dev)
    assert n.shape == () and abs(n.item() - ref) <= 2.0 ** -24 * ref * 1.01
    for max_norm in (0.5 * ref, 2 * ref, 0.0):
        scale = min(1.0, max_norm / (ref + EPS))
        for out_dtype in (None, torch.bfloat16, torch.float32):
            out = [torch.full_like(t, 7, dtype=out_dtype or t.dtype) for t in dev]
            got = M.clip_grad_norm(dev, max_norm, out=out)
            assert torch.equal(got, n)
            for o, t in zip(out, host):
                check(o, t, scale, out_dtype or t.dtype)
        work = [t.clone() for t in dev]
        assert torch.equal(M.clip_grad_norm(work, max_norm), n)
        for o, t in zip(work, host):
            check(o, t, scale, t.dtype)
            if scale == 1.0:
                assert torch.equal(o.cpu(), t)


def test_odd_addresses(M):
    """Views that start at any element of a buffer, and whose neighbours stay as they are."""
    import torch
    for dt, sizes in ((torch.bfloat16, [1, 3, 9, 255, 70001]), (torch.float32, [1, 2, 5, 33, 70003])):
        buf = torch.randn(sum(sizes) + 2 * len(sizes) + 1, device="cuda").to(dt)
        before = buf.clone()
        views, at = [], 1
        for n in sizes:
            views.append(buf[at : at + n])
            at += n + 2
        host = [v.cpu().clone() for v in views]
        ref = norm64(host)
        n = M.clip_grad_norm(views, 1.0)
        assert abs(n.item() - ref) <= 2.0 ** -24 * ref * 1.01
        keep = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
        at = 1
        for v, h in zip(views, host):
            check(v, h, min(1.0, 1.0 / (ref + EPS)), dt)
            keep[at : at + v.numel()] = False
            at += v.numel() + 2
        assert torch.equal(buf[keep], before[keep])


def test_extreme_values(M):
    """Squares that overflow or vanish in FP32, subnormal gradients, zeros, NaN and infinities."""
    import torch
    for v in (3e38, 1e30, 1e-30, 1e-40, 2.0 ** -149):
        t = torch.full((1000,), v, device="cuda")
        ref = float(t[0].double()) * math.sqrt(1000.0)
        n = M.grad_norm([t]).item()
        if ref > 3.4e38:
            assert n == math.inf
        else:
            assert abs(n - ref) <= 2.0 ** -24 * ref * 1.01 + 2.0 ** -150
    out = torch.empty(1000, device="cuda")
    big = torch.full((1000,), 3e37, device="cuda")
    M.clip_grad_norm([big], 1.0, out=[out])
    assert (out.double() * math.sqrt(1000.0) - 1.0).abs().max() < 1e-6
    z = torch.zeros(100, device="cuda")
    assert M.clip_grad_norm([z], 1.0).item() == 0.0 and not z.any()
    t = torch.ones(100, device="cuda")
    t[5] = math.nan
    assert math.isnan(M.clip_grad_norm([t, z], 1.0).item()) and t.isnan().all() and z.isnan().all()
    t, u = torch.ones(100, device="cuda"), torch.ones(9, dtype=torch.bfloat16, device="cuda")
    t[7] = math.inf
    assert M.clip_grad_norm([t, u], 1.0).item() == math.inf
    assert t[7].isnan() and not t[:7].any() and not u.any()


def test_same_bits_every_time(M):
    import torch
    dev = [t.cuda() for t in make([300000, 70001, 5] * 50, 4)]
    first = M.grad_norm(dev)
    for _ in range(3):
        assert torch.equal(M.grad_norm(dev), first)


def test_captured_clip(M):
    """A captured call clips by each replay's own norm."""
    import torch
    host = [make([70000, 33, 5], s, std=10.0 ** s) for s in range(4)]
    dev = [t.cuda() for t in host[0]]
    norm = torch.empty(1, device="cuda")
    M.clip_grad_norm([t.clone() for t in dev], 3.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.clip_grad_norm(dev, 3.0, norm=norm)
    for h in host:
        for d, t in zip(dev, h):
            d.copy_(t)
        ref = norm64(h)
        graph.replay()
        torch.cuda.synchronize()
        assert abs(norm.item() - ref) <= 2.0 ** -24 * ref * 1.01
        for d, t in zip(dev, h):
            check(d, t, min(1.0, 3.0 / (ref + EPS)), t.dtype)


def test_streams_and_refusals(M):
    import torch
    a = torch.randn(1000, device="cuda")
    ref = M.grad_norm([a])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n = M.grad_norm([a], stream=side)
    side.synchronize()
    assert torch.equal(n, ref)
    b = torch.randn(10, 10, device="cuda")
    for fn, match in [
        (lambda: M.grad_norm([]), "empty"), (lambda: M.grad_norm([a, b.t()]), "contiguous"), (lambda: M.grad_norm([a, 3]), "tensor"),
        (lambda: M.grad_norm([a.half()]), "type"), (lambda: M.grad_norm([a, b.cpu()]), "GPU"),
        (lambda: M.clip_grad_norm([a], 1.0, out=[]), "out has 0"), (lambda: M.clip_grad_norm([a], 1.0, out=[b]), "elements"),
        (lambda: M.grad_norm([a], norm=torch.empty(2, device="cuda")), "norm must"),
    ]:
        with pytest.raises(ValueError, match=match):
            fn()
    for fn, match in [
        (lambda: M.clip_grad_norm([a], -1.0), "max_norm"), (lambda: M.clip_grad_norm([a], math.nan), "max_norm"),
        (lambda: M.clip_grad_norm([a], 1.0, eps=-1.0), "eps"), (lambda: M.clip_grad_norm([a, a], 1.0), "overlap"),
        (lambda: M.clip_grad_norm([a[:10], a[10:20]], 1.0, out=[a[100:110], a[105:115]]), "overlap"),
        (lambda: M.clip_grad_norm([a[:10], a[10:20]], 1.0, out=[a[10:20], a[100:110]]), "overlap"),
        (lambda: M.grad_norm([a], norm=a[3:4]), "overlap"),
        (lambda: M.grad_norm([a], workspace=torch.empty(7, dtype=torch.uint8, device="cuda")), "workspace of 16"),
    ]:
        with pytest.raises(M.MgsError, match=match):
            fn()
    assert torch.equal(M.grad_norm([a, a]), torch.tensor(math.sqrt(2 * (a.double() ** 2).sum().item()), device="cuda"))
