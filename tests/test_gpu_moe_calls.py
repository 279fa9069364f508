"""The routing calls at the edges of what they take, on the device: rows past the caches and past 32-bit
offsets, tensors without elements, scores that underflow, streams and what is allocated for them."""

import numpy as np
import pytest

from helpers import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import moe_grouped_scaled_amd as M
    return M


def _picks(rng, t, k, e):
    """k distinct experts a token, a twentieth of the slots without one."""
    idx = np.argsort(rng.random((t, e)), axis=1)[:, :k].astype(np.int32)
    idx[rng.random((t, k)) < 0.05] = -1
    return idx


# 128 MiB of rows and more take the accesses that bypass the caches: widths that are no multiple of a workgroup's
# reach, every bound of topk, and one width that goes in single elements.  Sums of k products, each up to 2 in
# size, in FP32 in slot order against 64 bits: k roundings of 2^-24 of a partial sum up to 2 k, then one
# rounding of the result to its type.
@pytest.mark.parametrize("t,k,h,dtype", [(9000, 2, 4104, "bf16"), (5001, 4, 2056, "f32"), (3000, 16, 1608, "bf16"), (9000, 8, 1001, "bf16")])
def test_rows_far_larger_than_the_caches(M, t, k, h, dtype):
    import torch
    rng = np.random.default_rng(t)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    e = 33
    idx = to_dev(_picks(rng, t, k, e))
    gen = torch.Generator(device="cuda").manual_seed(t)
    x = torch.randn((t, h), generator=gen, device="cuda").clamp_(-2, 2).to(dt)
    w = torch.rand((t, k), generator=gen, device="cuda")
    rows = torch.full((t * k, h), 7.0, dtype=dt, device="cuda")
    rw = torch.full((t * k,), -1.0, device="cuda")
    row, splits = M.moe_dispatch(idx, e, x, rows, weights=w, row_weights=rw)
    used = int(splits.sum())
    live = row >= 0
    assert used == int(live.sum()) and used < t * k
    slot = live.nonzero()
    at = row[live].long()
    assert torch.equal(rows[at], x[slot[:, 0]]) and torch.equal(rw[at], w[live])
    assert bool((rows[used:] == 7.0).all()) and bool((rw[used:] == -1.0).all())

    def sums(r, weights):  # 64-bit, a thousand tokens at a time
        out = torch.empty((t, h), dtype=torch.float64, device="cuda")
        for t0 in range(0, t, 1000):
            n = row[t0:t0 + 1000]
            v = r[n.clamp(min=0).long()].double() * (n >= 0).double()[..., None]
            out[t0:t0 + 1000] = (v * weights[t0:t0 + 1000].double()[..., None] if weights is not None else v).sum(1)
        return out

    half = torch.finfo(dt).eps / 2
    for weights in (w, None):
        y, want = M.moe_combine(row, rows, weights=weights), sums(rows, weights)
        err = 2 * k * k * 2.0 ** -24
        assert bool(((y.double() - want).abs() <= (want.abs() + err) * half * 1.01 + err).all())
    dx, _ = M.moe_dispatch_bwd(row, rows)
    assert torch.equal(dx, y)
    drows = torch.full_like(rows, 7.0)
    dw = M.moe_combine_bwd(row, x, drows, rows=rows, weights=w)
    p = (x[slot[:, 0]].double() * w[live].double()[:, None])
    assert bool(((drows[at].double() - p).abs() <= p.abs() * (half * 1.01 + 2.0 ** -24)).all())
    assert bool((drows[used:] == 7.0).all()) and bool((dw[~live] == 0).all())
    # rows[at] is x: <dy, rows> is |x|^2, positive terms only, h roundings at most
    want = (x.double() ** 2).sum(1)[slot[:, 0]]
    assert bool(((dw[live].double() - want).abs() <= want * h * 2.0 ** -24).all())
    plain = torch.full_like(rows, 7.0)
    M.moe_combine_bwd(row, x, plain)
    assert torch.equal(plain, rows)


def test_offsets_past_32_bits(M):
    """4.4 G bytes of rows, 2.2 G elements: every offset of the last rows passes 2^31 elements."""
    import torch
    t, k, e, h = 4200, 4, 3, 131072
    idx = torch.full((t, k), -1, dtype=torch.int32, device="cuda")
    idx[:, 0], idx[:, 1], idx[:, 3] = 2, 0, 1
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((t, h), generator=gen, device="cuda", dtype=torch.bfloat16)
    rows = torch.full((t * k, h), 7.0, dtype=torch.bfloat16, device="cuda")
    row, splits = M.moe_dispatch(idx, e, x, rows)
    assert splits.tolist() == [t, t, t] and (3 * t) * h < 2 ** 31 < t * k * h
    want = torch.arange(t, dtype=torch.int32, device="cuda")
    assert torch.equal(row[:, 1], want) and torch.equal(row[:, 3], want + t) and torch.equal(row[:, 0], want + 2 * t)
    # the same rows again, moved to the end of the buffer, past 2^31 elements
    back = torch.where(row >= 0, row + t, row)
    rows.fill_(7.0)
    M.moe_combine_bwd(back, x, rows)
    for c in range(3):
        assert torch.equal(rows[(c + 1) * t:(c + 2) * t], x)
    assert bool((rows[:t] == 7.0).all())
    y = M.moe_combine(back, rows, weights=torch.ones((t, k), device="cuda") * 0.5)
    assert torch.equal(y, (1.5 * x.float()).to(torch.bfloat16))
    dw = M.moe_combine_bwd(back, x, rows=rows)
    n = (x.float() ** 2).sum(1, dtype=torch.float64)
    # h positive terms, summed by 256 threads and then over them: at most h / 256 + 10 roundings a term
    assert bool(((dw[:, [0, 1, 3]].double() - n[:, None]).abs() <= n[:, None] * (h / 256 + 10) * 2.0 ** -24).all())


def test_tensors_without_elements(M):
    import torch
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    bf = lambda *s: torch.full(s, 3.0, dtype=torch.bfloat16, device="cuda")
    f = lambda *s: torch.full(s, 3.0, device="cuda")
    for rows in (bf(0, 64), bf(5, 64)):
        rw = f(rows.shape[0])
        row, splits = M.moe_dispatch(i32(0, 2), 8, bf(0, 64), rows, weights=f(0, 2), row_weights=rw)
        assert row.shape == (0, 2) and splits.tolist() == [0] * 8 and bool((rows == 3).all()) and bool((rw == 3).all())
        assert M.moe_combine(row, rows).shape == (0, 64)
        dx, dw = M.moe_dispatch_bwd(row, rows, drow_weights=rw)
        assert dx.shape == (0, 64) and dw.shape == (0, 2)
        assert M.moe_combine_bwd(row, bf(0, 64), rows, rows=None) is None
    none = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    empty = bf(0, 64)
    assert bool((M.moe_combine(none, empty, weights=f(4, 2)) == 0).all())
    dx, dw = M.moe_dispatch_bwd(none, empty, drow_weights=f(0))
    assert bool((dx == 0).all()) and bool((dw == 0).all())
    assert M.moe_combine_bwd(none, bf(4, 64), empty) is None
    assert bool((M.moe_combine_bwd(none, bf(4, 64), empty.clone(), rows=empty) == 0).all())


def test_sigmoid_scores_near_the_smallest_numbers(M):
    """Scores of logits down to -100 are subnormal FP32 numbers, steps of 2^-149; their shares are as close as that
    and a few roundings (expf 2 steps, sum, quotient) allow, and the gradient's scores are the same."""
    import torch
    x = np.array([[-85.0, -86.0, -200.0, -300.0], [-90.0, -90.5, -91.0, -400.0], [-100.0, -99.0, -101.0, -98.0]], np.float32)
    x = np.concatenate([x, -x])
    s = 1 / (1 + np.exp(-x.astype(np.float64)))
    idx, w = M.moe_route(to_dev(x), 2, score="sigmoid", renormalize=True)
    p = np.take_along_axis(s, idx.cpu().numpy(), 1)
    want = p / p.sum(1, keepdims=True)
    tol = (2.0 ** -149 / p).max(1, keepdims=True) * 4 + 8 * 2.0 ** -24
    assert np.all(np.abs(w.cpu().numpy() - want) <= tol * want)
    g = torch.tensor([[1.0, -1.0]] * len(x), device="cuda")
    dl = M.moe_route_bwd(to_dev(x), idx, g, score="sigmoid", renormalize=True).cpu().numpy()
    picked = np.take_along_axis(dl, idx.cpu().numpy(), 1)
    q = 1 / (1 + np.exp(np.take_along_axis(x, idx.cpu().numpy(), 1).astype(np.float64)))
    wg = 2 * want[:, :1] * want[:, 1:] * np.array([[1.0, -1.0]]) * q
    assert np.all(np.abs(picked - wg) <= 4 * (tol + 2.0 ** -149 / q) * np.abs(wg))


def _stream_of(t):
    import torch
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not in the allocator's segments")


def test_what_a_call_allocates_belongs_to_its_stream(M):
    import torch
    rng = np.random.default_rng(0)
    logits = to_dev(rng.standard_normal((3000, 16)).astype(np.float32))
    x = torch.randn((3000, 64), device="cuda").to(torch.bfloat16)
    s = torch.cuda.Stream()

    def run(stream):
        rows = torch.zeros((6000, 64), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        idx, w = M.moe_route(logits, 2, stream=stream)
        row, splits = M.moe_dispatch(idx, 16, x, rows, stream=stream)
        y = M.moe_combine(row, rows, weights=w, stream=stream)
        drows = torch.zeros_like(rows)
        torch.cuda.synchronize()
        dw = M.moe_combine_bwd(row, x, drows, rows=rows, weights=w, stream=stream)
        dx, _ = M.moe_dispatch_bwd(row, drows, stream=stream)
        dl = M.moe_route_bwd(logits, idx, dw, stream=stream)
        torch.cuda.synchronize()
        return idx, w, row, splits, y, dw, dx, dl

    want = run(None)
    for stream, handle in ((s, s.cuda_stream), (s.cuda_stream, s.cuda_stream), (0, 0)):
        got = run(stream)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert all(_stream_of(t) == handle for t in got)


def test_two_streams_at_once(M):
    """Two dispatches with their sort's scratch in flight together."""
    import torch
    rng = np.random.default_rng(5)
    cases = [(to_dev(_picks(rng, 20000, 4, 64)), torch.randn((20000, 256), device="cuda").to(torch.bfloat16)) for _ in range(2)]
    want = []
    for idx, x in cases:
        rows = torch.zeros((80000, 256), dtype=torch.bfloat16, device="cuda")
        want.append((*M.moe_dispatch(idx, 64, x, rows), rows))
    outs = [torch.zeros((80000, 256), dtype=torch.bfloat16, device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(8):
        got = [M.moe_dispatch(idx, 64, x, rows, stream=s) for (idx, x), rows, s in zip(cases, outs, streams)]
    torch.cuda.synchronize()
    for (row, splits, rows), (r2, s2), out in zip(want, got, outs):
        assert torch.equal(row, r2) and torch.equal(splits, s2) and torch.equal(rows, out)


def test_a_stream_of_another_device_is_refused(M):
    import types
    import torch
    logits = torch.zeros((4, 8), device="cuda")
    with pytest.raises(ValueError, match="the stream is on"):
        M.moe_route(logits, 2, stream=types.SimpleNamespace(device=torch.device("cuda", 7), cuda_stream=0))
