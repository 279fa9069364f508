"""GPU parity of the router, the dispatch, the combine and their gradients, and of the layer they form with
the expert MLP, against 64-bit definitions written here.

Tolerances (u = 2^-24, the FP32 unit roundoff).  Experts, rows, split sizes and copied rows are exact.
  weights   exp of a difference d: the subtraction's rounding moves it by |d| u, the function by at most 2 u;
            a sum of E terms E u, a division and the scale 2 u: (|d| + E + 8) 2 u relative
  dlogits   products of such weights and sums over topk and E of them: (2 |d| + 2 E + 4 k + 24) 2 u of
            p_e (|g_e| + sum p |g|), before a BF16 rounding of half a step, 2^-8 of the value
  sums      n terms in FP32 in any order: (n + 2) u times the sum of magnitudes, plus the rounding of
            the result (2^-8 for BF16, 2^-24 for FP32)
"""

import itertools

import numpy as np
import pytest

import workloads
from tests.helpers import bf16_f64, bf16_host, f32, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def M():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_scaled_amd
    return moe_grouped_scaled_amd


# ------------------------------------------------------------------------------------------ router


def _logits(rng, t, e, dtype, masked):
    x = rng.standard_normal((t, e)).astype(np.float32) * 1.5
    if masked:
        x[rng.random((t, e)) < 0.3] = -np.inf
        x[rng.random(t) < 0.1] = -np.inf                 # tokens without any expert
        x[rng.random((t, e)) < 0.05] = -3.0e38           # the lowest values are there, if far away
        x[rng.random((t, e)) < 0.05] = 0.0
        x[rng.random((t, e)) < 0.05] = -0.0              # equal to 0: the lower expert first
    if dtype == "bf16":
        return to_dev_bf16(workloads.bf16_bits(x)), workloads.bf16_to_f32(workloads.bf16_bits(x)).astype(np.float64)
    return to_dev(x), x.astype(np.float64)


def _route64(x, k, score, renorm, scale):
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    vals = np.take_along_axis(x, order, 1)
    live = vals > -np.inf
    idx = np.where(live, order, -1)
    top = np.where(np.isfinite(x).any(1), x.max(1), 0.0)[:, None]
    if score == "softmax":
        z = np.exp(x - top)
        p = z / np.maximum(z.sum(1, keepdims=True), 1e-300)
        d = np.minimum(top - vals, 110.0)
    else:
        p = 1.0 / (1.0 + np.exp(np.minimum(-x, 709.0)))
        d = np.zeros_like(vals)
    w = np.where(live, np.take_along_axis(p, order, 1), 0.0)
    if renorm:
        s = w.sum(1, keepdims=True)
        w = np.where(s > 0, w / np.where(s > 0, s, 1.0), 0.0)
    return idx, order, live, p, scale * w, np.where(live, d, 0.0)


def _grad64(x, order, live, p, g, score, renorm, scale):
    w = np.where(live, np.take_along_axis(p, order, 1), 0.0)
    g = np.where(live, g, 0.0) * scale
    if renorm and score == "softmax":
        # the softmax over the picked ones alone: exactly 0 elsewhere
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
        dx = np.zeros_like(p)
        np.put_along_axis(dx, order, w * (w[:, None, :] * (g[:, :, None] - g[:, None, :])).sum(2), 1)
        return dx
    if renorm:
        s = np.maximum(w.sum(1, keepdims=True), 1e-300)
        g = np.where(live, (g - (g * w).sum(1, keepdims=True) / s) / s, 0.0)
    gp = np.zeros_like(p)
    np.put_along_axis(gp, order, g, 1)
    if score == "softmax":
        return p * (gp - (gp * p).sum(1, keepdims=True))
    return gp * p * (1.0 - p)


ROUTES = [(1, 1, 1), (1, 8, 2), (5, 16, 16), (3, 17, 3), (130, 32, 4), (67, 61, 5), (64, 64, 8), (33, 128, 1), (50, 129, 6), (300, 256, 8), (9, 256, 16)]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("score,renorm", itertools.product(["softmax", "sigmoid"], [False, True]))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,e,k", ROUTES)
def test_route_and_gradient(M, t, e, k, dtype, score, renorm, masked):
    import torch
    rng = np.random.default_rng(t * 1000 + e + k)
    dev, x = _logits(rng, t, e, dtype, masked)
    scale = 1.0 if e % 2 else 2.5
    idx, order, live, p, w, d = _route64(x, k, score, renorm, scale)
    got_i, got_w = M.moe_route(dev, k, score=score, renormalize=renorm, scale=scale)
    assert np.array_equal(got_i.cpu().numpy(), idx)
    assert np.all(np.abs(f32(got_w) - w) <= (np.max(d, 1, keepdims=True) + e + 8) * 2 * U * w + 1e-37)
    # a row stride, and outputs given
    wide = torch.full((t, e + 5), 9.0, dtype=dev.dtype, device="cuda")
    wide[:, 2:e + 2] = dev
    again_i, again_w = torch.empty_like(got_i), torch.empty_like(got_w)
    M.moe_route(wide[:, 2:e + 2], k, score=score, renormalize=renorm, scale=scale, expert_idx=again_i, weights=again_w)
    assert torch.equal(again_i, got_i) and torch.equal(again_w, got_w)
    g = rng.standard_normal((t, k)).astype(np.float32)
    ref = _grad64(x, order, live, p, g.astype(np.float64), score, renorm, scale)
    dl = M.moe_route_bwd(dev, got_i, to_dev(g), score=score, renormalize=renorm, scale=scale)
    assert dl.dtype == dev.dtype
    gs = np.abs(np.where(live, g, 0.0) * scale)
    pw = np.abs(w) / scale
    size = np.zeros_like(p)
    np.put_along_axis(size, order, np.where(live, pw * gs, 0.0), 1)
    size += (np.abs(p) if score == "softmax" and not renorm else (size > 0)) * (pw * gs).sum(1, keepdims=True)
    if renorm:  # w_e sum_i w_i |g_e - g_i|
        sz = np.zeros_like(p)
        np.put_along_axis(sz, order, np.where(live, pw * (gs + (pw * gs).sum(1, keepdims=True)), 0.0), 1)
        size = sz
    bound = (2 * np.max(d, 1, keepdims=True) + 2 * e + 4 * k + 24) * 2 * U * size + 1e-36
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * np.abs(ref)
    got = f32(dl.float())
    assert np.all(np.abs(got - ref) <= bound)
    into = torch.full((t, e + 3), 4.0, dtype=dev.dtype, device="cuda")
    M.moe_route_bwd(wide[:, 2:e + 2], got_i, to_dev(g), score=score, renormalize=renorm, scale=scale, dlogits=into[:, :e])
    assert torch.equal(into[:, :e], dl) and bool((into[:, e:] == 4.0).all())


@pytest.mark.parametrize("score,renorm", itertools.product(["softmax", "sigmoid"], [False, True]))
def test_route_gradient_against_differences(M, score, renorm):
    """Central differences of the 64-bit weights, step 1e-5: truncation below 1e-10, cancellation 1e-11."""
    t, e, k = 6, 12, 3
    rng = np.random.default_rng(5)
    x = rng.standard_normal((t, e)).astype(np.float32).astype(np.float64)
    g = rng.standard_normal((t, k)).astype(np.float32)
    idx, order, live, p, _, _ = _route64(x, k, score, renorm, 1.0)

    def loss(v):
        q = 1.0 / (1.0 + np.exp(-v)) if score == "sigmoid" else np.exp(v) / np.exp(v).sum(1, keepdims=True)
        w = np.take_along_axis(q, order, 1)
        return ((w / w.sum(1, keepdims=True) if renorm else w) * g).sum(1)

    num = np.zeros_like(x)
    for j in range(e):
        h = np.zeros_like(x)
        h[:, j] = 1e-5
        num[:, j] = (loss(x + h) - loss(x - h)) / 2e-5
    got = f32(M.moe_route_bwd(to_dev(x.astype(np.float32)), to_dev(idx.astype(np.int32)), to_dev(g), score=score, renormalize=renorm))
    # size 1 weights and gradients: the FP32 bound above with E = 12, k = 3, |d| < 8
    assert np.max(np.abs(got - num)) <= 100 * 2 * U * np.max(np.abs(g)) * k + 1e-9


def test_route_infinities_and_nan(M):
    x = np.zeros((6, 20), np.float32)
    x[0, 7] = np.nan                       # picked first, and the weights say so
    x[1, 3] = np.inf
    x[2] = -np.inf
    x[3, 1:] = -np.inf                     # one expert available for two choices
    x[4] = -3.0e38                         # lowest, but available
    x[5, 4], x[5, 9] = 1.0, 1.0            # a tie
    for score in ("softmax", "sigmoid"):
        idx, w = M.moe_route(to_dev(x), 2, score=score, renormalize=True)
        idx, w = idx.cpu().numpy(), f32(w)
        assert idx.tolist() == [[7, 0], [3, 0], [-1, -1], [0, -1], [0, 1], [4, 9]]
        assert np.isnan(w[0]).any() and (np.isnan(w[1]).any() or score == "sigmoid")
        assert w[2].tolist() == [0.0, 0.0] and w[3].tolist() == [1.0, 0.0]
        assert w[4].tolist() == ([0.5, 0.5] if score == "softmax" else [0.0, 0.0]) and w[5].tolist() == [0.5, 0.5]
        for renorm in (False, True):
            d = f32(M.moe_route_bwd(to_dev(x), to_dev(idx.astype(np.int32)), to_dev(np.ones((6, 2), np.float32)), score=score, renormalize=renorm))
            assert not d[2].any() and np.isfinite(d[2:]).all()
            assert not d[3, 1:].any()


# ------------------------------------------------------------------------------------------ dispatch


def _experts(rng, t, k, e, dropped):
    idx = np.stack([rng.permutation(e)[:k] if e >= k else rng.integers(0, e, k) for _ in range(t)]) if t else np.zeros((0, k))
    idx = idx.astype(np.int32)
    if dropped:
        idx[rng.random((t, k)) < 0.25] = -1
        idx[rng.random((t, k)) < 0.02] = e                  # outside: no expert either
        idx[rng.random((t, k)) < 0.02] = 2 ** 31 - 1
    return idx


def _sorted64(idx, e):
    flat = idx.reshape(-1).astype(np.int64)
    ok = (flat >= 0) & (flat < e)
    order = np.argsort(np.where(ok, flat, e), kind="stable")
    row = np.empty(flat.size, np.int64)
    row[order] = np.arange(flat.size)
    return np.where(ok, row, -1).reshape(idx.shape), np.bincount(flat[ok], minlength=e)[:e]


MOVES = [(1, 1, 1, 1), (1, 2, 4, 64), (3, 2, 16, 4096), (7, 3, 61, 1001), (64, 8, 256, 128), (257, 1, 5, 72), (340, 6, 200, 40),
         (1000, 4, 32, 200), (1, 16, 256, 7168), (700, 16, 16, 24)]


def _rows(rng, shape, dtype):
    if dtype == "bf16":
        b = workloads.normal_bf16(rng, shape)
        return to_dev_bf16(b), bf16_f64(b)
    v = rng.standard_normal(shape).astype(np.float32)
    return to_dev(v), v.astype(np.float64)


@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,k,e,h", MOVES)
def test_dispatch_combine_and_gradients(M, t, k, e, h, dtype, dropped):
    import torch
    rng = np.random.default_rng(t + k + e + h)
    idx = _experts(rng, t, k, e, dropped)
    row64, counts = _sorted64(idx, e)
    there = row64 >= 0
    m, used = t * k, int(there.sum())
    half = 2.0 ** -8 if dtype == "bf16" else U
    xd, x = _rows(rng, (t, h), dtype)
    w = rng.random((t, k), dtype=np.float32)
    rows = torch.full((m + 3, h), 7.0, dtype=xd.dtype, device="cuda")
    rw = torch.full((m + 3,), 7.0, device="cuda")
    row, splits = M.moe_dispatch(to_dev(idx), e, xd, rows, weights=to_dev(w), row_weights=rw)
    assert np.array_equal(row.cpu().numpy(), row64) and np.array_equal(splits.cpu().numpy(), counts)
    want, want_w = np.full((m + 3, h), 7.0), np.full(m + 3, 7.0)
    tok = np.repeat(np.arange(t), k).reshape(t, k)
    want[row64[there]] = x[tok[there]]
    want_w[row64[there]] = w[there]
    assert np.array_equal(f32(rows.float()), want) and np.array_equal(f32(rw), want_w)
    # only the sort; a row stride and an unaligned start
    only, s2 = M.moe_dispatch(to_dev(idx), e)
    assert torch.equal(only, row) and torch.equal(s2, splits)
    wide = torch.zeros((t, h + 3), dtype=xd.dtype, device="cuda")
    wide[:, 1:h + 1] = xd
    rows2 = torch.full((m + 3, h), 7.0, dtype=xd.dtype, device="cuda")
    M.moe_dispatch(to_dev(idx), e, wide[:, 1:h + 1], rows2)
    assert torch.equal(rows2, rows)
    # combine, with weights and without
    outd, out = _rows(rng, (m + 3, h), dtype)
    safe = np.maximum(row64, 0)
    for weights in (w, None):
        ww = (np.ones((t, k)) if weights is None else w.astype(np.float64)) * there
        ref = np.einsum("tk,tkh->th", ww, out[safe])
        size = np.einsum("tk,tkh->th", ww, np.abs(out[safe]))
        y = M.moe_combine(row, outd, weights=None if weights is None else to_dev(w))
        assert np.all(np.abs(f32(y.float()) - ref) <= (k + 2) * U * size + half * np.abs(ref))
        into = torch.full((t, h + 3), 5.0, dtype=xd.dtype, device="cuda")
        M.moe_combine(row, outd, weights=None if weights is None else to_dev(w), y=into[:, 1:h + 1])
        assert torch.equal(into[:, 1:h + 1], y) and bool((into[:, :1] == 5.0).all()) and bool((into[:, h + 1:] == 5.0).all())
        # gradient of the combine
        dyd, dy = _rows(rng, (t, h), dtype)
        drows = torch.full((m + 3, h), 7.0, dtype=xd.dtype, device="cuda")
        dw = M.moe_combine_bwd(row, dyd, drows, rows=outd, weights=None if weights is None else to_dev(w))
        dref = np.full((m + 3, h), 7.0)
        dref[row64[there]] = (dy[tok] * ww[:, :, None])[there]
        gap = np.abs(f32(drows.float()) - dref)
        assert np.all(gap <= (half if weights is not None else 0.0) * np.abs(dref) * (1 + 2 ** -8) + 1e-44)
        wref = np.einsum("th,tkh->tk", dy, out[safe]) * there
        wsize = np.einsum("th,tkh->tk", np.abs(dy), np.abs(out[safe])) * there
        assert np.all(np.abs(f32(dw) - wref) <= (h + 2) * U * wsize)
        alone = torch.full((m + 3, h), 7.0, dtype=xd.dtype, device="cuda")
        assert M.moe_combine_bwd(row, dyd, alone, weights=None if weights is None else to_dev(w)) is None
        assert torch.equal(alone, drows)
        assert torch.equal(M.moe_combine_bwd(row, dyd, rows=outd, weights=None if weights is None else to_dev(w)), dw)
    # gradient of the dispatch
    gp = rng.standard_normal(m + 3).astype(np.float32)
    dx, dw = M.moe_dispatch_bwd(row, outd, drow_weights=to_dev(gp))
    ref, size = (out[safe] * there[:, :, None]).sum(1), (np.abs(out[safe]) * there[:, :, None]).sum(1)
    assert np.all(np.abs(f32(dx.float()) - ref) <= (k + 2) * U * size + half * np.abs(ref))
    assert np.array_equal(f32(dw), np.where(there, gp[safe], 0.0))
    dx2, none = M.moe_dispatch_bwd(row, outd)
    assert none is None and torch.equal(dx2, dx)


@pytest.mark.parametrize("t,k,e", [(0, 2, 8), (2048, 1, 7), (2049, 1, 256), (5000, 3, 64), (16384, 8, 256), (40000, 4, 33), (70001, 2, 1)])
def test_sort_over_chunk_borders(M, t, k, e):
    rng = np.random.default_rng(t)
    idx = rng.integers(-1, e + 1, (t, k)).astype(np.int32)
    row64, counts = _sorted64(idx, e)
    row, splits = M.moe_dispatch(to_dev(idx), e)
    assert np.array_equal(row.cpu().numpy(), row64) and np.array_equal(splits.cpu().numpy(), counts)


def test_one_expert_takes_all_and_the_same_expert_twice(M):
    idx = np.full((900, 4), 3, np.int32)
    row, splits = M.moe_dispatch(to_dev(idx), 9)
    assert np.array_equal(row.cpu().numpy().reshape(-1), np.arange(3600)) and splits.tolist() == [0, 0, 0, 3600] + [0] * 5


def test_rows_outside_count_as_none(M):
    """A row number outside the rows (as after a buffer of another step) is no row, in every call."""
    import torch
    row = to_dev(np.array([[0, 5], [-7, 2], [2 ** 31 - 1, 1]], np.int32))
    rows, _ = _rows(np.random.default_rng(0), (3, 16), "bf16")
    y = M.moe_combine(row, rows)
    assert torch.equal(y, rows[torch.tensor([0, 2, 1], device="cuda")])
    drows = torch.full((3, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = M.moe_combine_bwd(row, y, drows, rows=rows)
    assert torch.equal(drows, rows) and dw.cpu().numpy()[[0, 1, 2], [1, 0, 0]].tolist() == [0.0, 0.0, 0.0]


def test_another_stream(M):
    import torch
    rng = np.random.default_rng(1)
    x, _ = _rows(rng, (500, 512), "bf16")
    logits = to_dev(rng.standard_normal((500, 16)).astype(np.float32))
    idx, w = M.moe_route(logits, 2)
    rows = torch.zeros((1000, 512), dtype=torch.bfloat16, device="cuda")
    row, splits = M.moe_dispatch(idx, 16, x, rows)
    y = M.moe_combine(row, rows, weights=w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    rows2 = torch.zeros_like(rows)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        idx2, w2 = M.moe_route(logits, 2)
        row2, splits2 = M.moe_dispatch(idx2, 16, x, rows2)
        y2 = M.moe_combine(row2, rows2, weights=w2)
    i3, w3 = M.moe_route(logits, 2, stream=s)
    s.synchronize()
    for a, b in ((idx, idx2), (w, w2), (row, row2), (splits, splits2), (rows, rows2), (y, y2), (idx, i3), (w, w3)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------ the layer

T, E, K, H, F = 150, 4, 2, 128, 128


def _layer(M, fmt, kind="srelu", seed=3, **kw):
    from moe_grouped_scaled_amd.expert_mlp import ExpertMLP
    rng = np.random.default_rng(seed)
    f_in = 2 * F if kind == "swiglu" else F
    d = dict(w1=workloads.normal_bf16(rng, (E, f_in, H), 0.05), w2=workloads.normal_bf16(rng, (E, H, F), 0.05),
             b1=workloads.normal_bf16(rng, (E, f_in), 0.05), b2=workloads.normal_bf16(rng, (E, H), 0.05))
    mlp = ExpertMLP(kind, fmt, *[to_dev_bf16(d[k]) for k in ("w1", "w2", "b1", "b2")], recompute=True, **kw)
    return M.MoELayer(mlp, K), d


def _layer_inputs(rng, masked=True):
    logits = rng.standard_normal((T, E)).astype(np.float32)
    if masked:
        logits[::17] = -np.inf
        logits[5::23, 1:] = -np.inf
        logits[:, 2] = -np.inf                        # an empty expert
    return to_dev_bf16(workloads.normal_bf16(rng, (T, H))), to_dev(logits), to_dev_bf16(workloads.normal_bf16(rng, (T, H)))


@pytest.mark.parametrize("fmt,kind", [("mxfp8", "srelu"), ("mxfp4", "srelu"), ("mxfp4", "swiglu"), ("nvfp4", "srelu")])
def test_layer_equals_its_parts_on_host_splits(M, fmt, kind):
    """The layer (device-resident split sizes, capacity layouts) against rows sorted by numpy and the
    expert MLP with host split sizes: bit for bit on rows and gradients of rows, and the sums per token
    recomputed in 64 bits from those."""
    import torch
    rng = np.random.default_rng(11)
    x, logits, dy = _layer_inputs(rng)
    layer, _ = _layer(M, fmt, kind)
    y = layer.forward(x, logits)
    g = layer.backward(dy)
    torch.cuda.synchronize()
    ref, _ = _layer(M, fmt, kind)
    idx, order, live, p, w, _ = _route64(f32(logits), K, "softmax", True, 1.0)
    row, counts = _sorted64(idx, E)
    there = row >= 0
    tok = np.repeat(np.arange(T), K).reshape(T, K)
    n = int(counts.sum())
    src = np.empty(n, np.int64)
    src[row[there]] = tok[there]
    probs = np.empty(n, np.float32)
    _, wd = M.moe_route(logits, K)
    probs[row[there]] = wd.cpu().numpy()[there]
    src = torch.from_numpy(src).cuda()
    y_rows = ref.mlp.forward(x[src].contiguous(), to_dev(probs), counts.tolist())
    want = ref.mlp.backward(dy[src].contiguous())
    torch.cuda.synchronize()
    for k in ("dw1", "dw2", "db1", "db2"):
        assert torch.equal(g[k], want[k]), k
    safe = np.maximum(row, 0)
    for got, rows in ((y, y_rows), (g["dx"], want["dx1"])):
        r = bf16_f64(bf16_host(rows))
        ref64, size = (r[safe] * there[:, :, None]).sum(1), (np.abs(r[safe]) * there[:, :, None]).sum(1)
        assert np.all(np.abs(bf16_f64(bf16_host(got)) - ref64) <= (K + 2) * U * size + 2.0 ** -8 * np.abs(ref64))
    dw = np.where(there, f32(want["dprobs"])[safe], 0.0)
    dref = _grad64(f32(logits), order, live, p, dw, "softmax", True, 1.0)
    size = np.abs(dw).sum(1, keepdims=True)
    assert np.all(np.abs(f32(g["dlogits"]) - dref) <= (2 * 8 + 2 * E + 4 * K + 24) * 4 * U * size + 1e-36)
    assert not f32(g["dlogits"])[::17].any() and not bf16_f64(bf16_host(y))[::17].any()


def test_layer_without_token_gradients(M):
    """With the token gradient not requested the logits still get theirs, the same bits."""
    import torch
    x, logits, dy = _layer_inputs(np.random.default_rng(12))
    full, _ = _layer(M, "mxfp8")
    part, _ = _layer(M, "mxfp8", grad_x1=False)
    full.forward(x, logits)
    part.forward(x, logits)
    a, b = full.backward(dy), part.backward(dy)
    assert "dx" not in b and torch.equal(a["dlogits"], b["dlogits"]) and torch.equal(a["dw1"], b["dw1"])


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_layer_graph_follows_the_routing(M, fmt):
    """One captured graph of the layer's step, replayed for routings A, B, C, A with eager work between the
    replays: every replay equals the eager step."""
    import torch
    rng = np.random.default_rng(13)
    cases = [_layer_inputs(rng, masked=i != 1) for i in range(3)]
    x, logits, dy = [t.clone() for t in cases[0]]
    layer, _ = _layer(M, fmt)

    def step(a, b, c):
        y = layer.forward(a, b)
        return dict(layer.backward(c), y=y)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(x, logits, dy)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(x, logits, dy)
    for i in (0, 1, 2, 0):
        ref = {k: v.clone() for k, v in step(*cases[i]).items()}
        torch.cuda.synchronize()
        for dst, src in zip((x, logits, dy), cases[i]):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        for k, v in ref.items():
            assert torch.equal(out[k], v), (i, k)
