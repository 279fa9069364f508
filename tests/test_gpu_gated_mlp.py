"""`GatedMLP`, its place in `MoELayer`, captured graphs, streams, and its gradients.

Bounds: every stage rounds to BF16 once (2^-8 at most, 2^-8 / sqrt(3) in the mean square of a uniform error), and each
rounding before an output reaches it through sums of many terms of independent error, so the relative 2-norm
of an output's error stays below the square root of the sum of the squares of its roundings, and below
sqrt(roundings) 2^-8 even if each error were at its bound.
"""

import math

import pytest

from test_gpu_gated import KINDS, LIMIT, ALPHA, BETA, act64, bounds, device_groups

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_scaled_amd as m
    return m


def params(e, h, f, seed, bias):
    import torch
    gen = torch.Generator().manual_seed(seed)
    bf = lambda *s, std: (torch.randn(s, generator=gen) * std).to(torch.bfloat16)
    w1, w2 = bf(e, 2 * f, h, std=h ** -0.5), bf(e, h, f, std=f ** -0.5)
    return w1, w2, (bf(e, 2 * f, std=0.3) if bias else None), (bf(e, h, std=0.3) if bias else None)


def step64(kind, splits, x, p, dy, w1, w2, b1, b2):
    """The block and its gradients in 64 bits."""
    import torch
    d = lambda t: None if t is None else t.double()
    x, p, dy, w1, w2, b1, b2 = map(d, (x, p, dy, w1, w2, b1, b2))
    f = w2.shape[2]
    o = dict(y=torch.zeros_like(dy), dx1=torch.zeros_like(x), dprobs=torch.zeros(x.shape[0], dtype=torch.float64),
             dw1=torch.zeros_like(w1), dw2=torch.zeros_like(w2), db1=torch.zeros(w1.shape[:2], dtype=torch.float64),
             db2=torch.zeros(w2.shape[:2], dtype=torch.float64))
    for g, at in bounds(splits):
        pre = x[at] @ w1[g].t() + (0 if b1 is None else b1[g])
        a, by_g, by_u, _, _ = act64(kind, pre[:, :f], pre[:, f:])
        s = 1.0 if p is None else p[at][:, None]
        o["y"][at] = (a * s) @ w2[g].t() + (0 if b2 is None else b2[g])
        da = dy[at] @ w2[g]
        dpre = torch.cat([da * s * by_g, da * s * by_u], 1)
        o["dprobs"][at] = (da * a).sum(1)
        o["dx1"][at], o["dw1"][g], o["dw2"][g] = dpre @ w1[g], dpre.t() @ x[at], dy[at].t() @ (a * s)
        o["db1"][g], o["db2"][g] = dpre.sum(0), dy[at].sum(0)
    return o


# roundings to BF16 that an output has seen (its own counted): pre kept in BF16, h, dpre, y, ...
ROUNDINGS = dict(y=2, dx1=3, dprobs=1, dw1=3, dw2=2, db1=2, db2=0)


def near(got, ref, what, extra=0):
    rel = ((got.double().cpu() - ref).norm() / ref.norm().clamp_min(1e-30)).item()
    n = ROUNDINGS[what] + extra
    assert rel <= (math.sqrt(n) * 2.0 ** -8 if n else 1e-5), (what, rel)


def run_step(mlp, splits, x, p, dy):
    y = mlp.forward(x, p, splits)
    g = mlp.backward(dy)
    if mlp.delay_wgrad:
        g.update(mlp.backward_dw())
    return dict(g, y=y)


@pytest.mark.parametrize("recompute,delay", [(False, False), (True, True)])
@pytest.mark.parametrize("bias,probs", [(True, True), (False, False)])
@pytest.mark.parametrize("kind", KINDS)
def test_step_against_64_bits(M, kind, bias, probs, recompute, delay):
    import torch
    splits, h, f = [37, 0, 130, 1], 136, 200
    w1, w2, b1, b2 = params(4, h, f, 1, bias)
    gen = torch.Generator().manual_seed(2)
    m = sum(splits)
    x, dy = torch.randn(m, h, generator=gen).to(torch.bfloat16), torch.randn(m, h, generator=gen).to(torch.bfloat16)
    p = torch.rand(m, generator=gen) + 0.25 if probs else None
    ref = step64(kind, splits, x, p, dy, w1, w2, b1, b2)
    dev = [None if t is None else t.cuda() for t in (w1, w2, b1, b2)]
    for dt in (torch.float32, torch.bfloat16):
        mlp = M.GatedMLP(kind, dev[0], dev[1], dev[2], dev[3], recompute=recompute, delay_wgrad=delay, limit=LIMIT, alpha=ALPHA,
                         beta=BETA, dw_dtype=dt, save_dtype=dt)
        got = run_step(mlp, splits, x.cuda(), None if p is None else p.cuda(), dy.cuda())
        assert got["dw1"].dtype == dt and got["dw2"].dtype == dt
        want = ["y", "dx1", "dprobs", "dw1", "dw2"] + (["db1", "db2"] if bias else [])
        assert set(got) == set(want)
        for name in want:
            # regenerated rows carry the rounding of [gate | up] too; kept in FP32 there is none
            if dt == torch.bfloat16:
                extra = 1 if recompute and name == "dw2" else 0
            else:
                extra = -1 if name in ("dx1", "dprobs", "dw1", "db1") else 0
            near(got[name], ref[name], name, extra=extra)


def test_gradients_against_differences(M):
    """The loss sum(dy * y) in 64 bits, moved along the gradients that the kernels return."""
    import torch
    splits, h, f, kind = [9, 20], 64, 72, "swiglu"
    w1, w2, b1, b2 = params(2, h, f, 3, True)
    gen = torch.Generator().manual_seed(4)
    m = sum(splits)
    x, dy = torch.randn(m, h, generator=gen).to(torch.bfloat16), torch.randn(m, h, generator=gen).to(torch.bfloat16)
    p = torch.rand(m, generator=gen) + 0.25
    mlp = M.GatedMLP(kind, *[t.cuda() for t in (w1, w2, b1, b2)])
    got = {k: v.double().cpu() for k, v in run_step(mlp, splits, x.cuda(), p.cuda(), dy.cuda()).items()}
    at = dict(dx1=x, dprobs=p, dw1=w1, dw2=w2, db1=b1, db2=b2)
    names = list(at)

    def loss(v):
        return (dy.double() * step64(kind, splits, v["dx1"], v["dprobs"], dy, v["dw1"], v["dw2"], v["db1"], v["db2"])["y"]).sum()

    for name in names:
        direction = got[name] / got[name].norm()
        eps = 1e-4 * max(1.0, at[name].double().norm().item())
        up, down = ({**{n: at[n].double() for n in names}, name: at[name].double() + s * eps * direction} for s in (1, -1))
        slope = ((loss(up) - loss(down)) / (2 * eps)).item()
        # the slope along the normed gradient is its norm, less the part of its error along it
        n = max(ROUNDINGS[name], 1)
        assert abs(slope - got[name].norm().item()) <= math.sqrt(n) * 2.0 ** -8 * got[name].norm().item() + 1e-6, name


@pytest.mark.parametrize("want", [dict(grad_fc1=False), dict(grad_fc2=False), dict(grad_x1=False, grad_probs=False),
                                  dict(grad_x1=False, grad_probs=False, grad_fc1=False),
                                  dict(grad_x1=False, grad_probs=False, grad_fc1=False, grad_fc2=False)])
@pytest.mark.parametrize("recompute", [False, True])
def test_partial_gradients_match_the_full_step(M, want, recompute):
    import torch
    splits, h, f = [20, 0, 45], 72, 88
    dev = [t.cuda() for t in params(3, h, f, 5, True)]
    gen = torch.Generator().manual_seed(6)
    x, dy = (torch.randn(65, h, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    p = torch.rand(65, generator=gen).cuda()
    full = run_step(M.GatedMLP("glu", *dev, recompute=recompute), splits, x, p, dy)
    part = run_step(M.GatedMLP("glu", *dev, recompute=recompute, **want), splits, x, p, dy)
    names = {"y"}
    for flag, keys in (("grad_x1", ["dx1"]), ("grad_probs", ["dprobs"]), ("grad_fc1", ["dw1", "db1"]), ("grad_fc2", ["dw2", "db2"])):
        if want.get(flag, True):
            names.update(keys)
    assert set(part) == names
    for k in names:
        assert torch.equal(part[k], full[k]), k


def test_accumulated_weight_gradients(M):
    import torch
    splits, h, f = [20, 0, 45], 72, 88
    dev = [t.cuda() for t in params(3, h, f, 7, False)[:2]]
    gen = torch.Generator().manual_seed(8)
    x, dy = (torch.randn(65, h, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True, grad_probs=False)
    mlp.forward(x, None, splits)
    mlp.backward(dy)
    one = mlp.backward_dw()
    dw1, dw2 = one["dw1"].clone(), one["dw2"].clone()
    mlp.forward(x, None, splits)
    mlp.backward(dy)
    mlp.backward_dw(dw1, dw2, accumulate=True)
    assert torch.equal(dw1, 2 * one["dw1"]) and torch.equal(dw2, 2 * one["dw2"])


def layer_case(e, h, f, tokens, seed, bias):
    import torch
    dev = [None if t is None else t.cuda() for t in params(e, h, f, seed, bias)]
    gen = torch.Generator().manual_seed(seed + 1)
    x, dy = (torch.randn(tokens, h, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    return dev, x, torch.randn(tokens, e, generator=gen).cuda(), dy


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("tokens", [0, 1, 67])
def test_layer_against_64_bits(M, tokens, bias):
    """MoELayer around the block: y = sum_j w_j block_j(x), and its gradients, from the definition."""
    import torch
    e, h, f, topk, kind = 5, 64, 104, 2, "swiglu"
    dev, x, logits, dy = layer_case(e, h, f, tokens, 9, bias)
    layer = M.MoELayer(M.GatedMLP(kind, *dev), topk)
    y = layer.forward(x, logits)
    g = layer.backward(dy)
    lg = logits.double().cpu().requires_grad_()
    leaf = {n: t.double().cpu().requires_grad_() for n, t in zip(("w1", "w2", "b1", "b2"), dev) if t is not None}
    xd = x.double().cpu().requires_grad_()
    top = lg.topk(topk, dim=1)
    w = torch.softmax(top.values, dim=1)
    out = torch.zeros(tokens, h, dtype=torch.float64)
    rows = []
    for j in range(topk):
        for t in range(tokens):
            k = top.indices[t, j]
            pre = leaf["w1"][k] @ xd[t] + (leaf["b1"][k] if bias else 0)
            a = pre[:f] * torch.sigmoid(pre[:f]) * pre[f:]
            rows.append((t, w[t, j] * (leaf["w2"][k] @ a + (leaf["b2"][k] if bias else 0))))
    if rows:
        out = out.index_add(0, torch.tensor([t for t, _ in rows]), torch.stack([v for _, v in rows]))
    assert y.shape == (tokens, h)
    assert set(g) == {"dx", "dlogits", "dw1", "dw2"} | ({"db1", "db2"} if bias else set())
    if not tokens:
        assert not g["dw1"].any() and not g["dw2"].any()
        return
    (out * dy.double().cpu()).sum().backward()
    rel = lambda a, b: ((a.double().cpu() - b).norm() / b.norm()).item()
    # at most five roundings between the inputs and any of these
    bound = math.sqrt(5) * 2.0 ** -8
    assert rel(y, out.detach()) < bound and rel(g["dx"], xd.grad) < bound and rel(g["dlogits"], lg.grad) < 2 * bound
    for n in leaf:
        assert rel(g["d" + n], leaf[n].grad) < bound, n


def test_captured_layer_follows_the_routing(M):
    """One captured forward and backward, replayed for other inputs and routings, equal to the eager step."""
    import torch
    e, h, f, topk, tokens = 4, 64, 72, 2, 33
    dev, x, logits, dy = layer_case(e, h, f, tokens, 11, True)
    layer = M.MoELayer(M.GatedMLP("swiglu", *dev), topk)

    def step():
        y = layer.forward(x, logits)
        return dict(layer.backward(dy), y=y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    gen = torch.Generator().manual_seed(12)
    for i in range(4):
        x.copy_(torch.randn(tokens, h, generator=gen))
        logits.copy_(torch.randn(tokens, e, generator=gen) + (torch.tensor([9.0, 0, 0, 0]) if i == 2 else 0))
        dy.copy_(torch.randn(tokens, h, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()}
        ref = step()
        for k in ref:
            assert torch.equal(got[k], ref[k]), (i, k)


def test_side_stream_and_stream_argument(M):
    import torch
    splits, h, f = [30, 12], 64, 72
    dev = [t.cuda() for t in params(2, h, f, 13, True)]
    x = torch.randn(42, h, device="cuda").to(torch.bfloat16)
    p = torch.rand(42, device="cuda")
    ref = M.grouped_gated_fwd("swiglu", splits, x, dev[0], dev[2], p)
    y = M.grouped_gemm_bf16("fprop", splits, ref, dev[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = M.grouped_gated_fwd("swiglu", splits, x, dev[0], dev[2], p)
        y2 = M.grouped_gemm_bf16("fprop", splits, got, dev[1])
    side.synchronize()
    assert torch.equal(got, ref) and torch.equal(y2, y)
    for s in (side, side.cuda_stream, 0):
        got = M.grouped_gated_fwd("swiglu", splits, x, dev[0], dev[2], p, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, ref)


def test_refusals_on_the_gpu(M):
    import torch
    w1, w2, b1, b2 = [t.cuda() for t in params(2, 64, 72, 14, True)]
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    big = torch.zeros(8 * 72 + 8, dtype=torch.bfloat16, device="cuda")
    for fn, match in [
        (lambda: M.grouped_gated_fwd("swiglu", [8], x, w1), "2 experts"),
        (lambda: M.grouped_gated_fwd("swiglu", [4, 4], x[:, :32].contiguous(), w1), "width"),
        (lambda: M.grouped_gated_fwd("swiglu", [4, 4], x, w1, h=big[:576].view(8, 72).float()), "type"),
        (lambda: M.grouped_gated_fwd("swiglu", [4, 4], x, w1, probs=torch.zeros(7, device="cuda")), "shape"),
        (lambda: M.grouped_gated_fwd("swiglu", [4, 3], x, w1), "rows"),
        (lambda: M.grouped_gated_fwd("swiglu", device_groups([4, 4], 16), x, w1), "capacity"),
        (lambda: M.GatedMLP("swiglu", w1, w2[:, :, :64].contiguous()), "shape"),
        (lambda: M.GatedMLP("swiglu", w1, w2, b1.float()), "type"),
        (lambda: M.GatedMLP("swiglu", w1, w2).backward(x), "without a forward"),
        (lambda: M.GatedMLP("swiglu", w1, w2).backward_dw(), "without a pending"),
    ]:
        with pytest.raises(ValueError, match=match):
            fn()
    with pytest.raises(M.MgsError, match="16-byte"):
        M.grouped_gated_fwd("swiglu", [4, 4], x, w1, h=big[1:577].view(8, 72))
