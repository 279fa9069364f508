"""The BF16 block, gradient clipping and the 4-bit block as they are used together: a layer is trained for some steps with
clipped gradients, its weights are quantized to 4 bits, and the layer serves with them.  Every part is held against 64 bits
from what the part before it returned, so that each tolerance is of one operator.
"""

import math

import pytest

from test_gpu_gated import UBF
from test_gpu_grad_clip import norm64
from test_gpu_w4 import values64

pytestmark = pytest.mark.gpu

E, H, F, TOPK, TOKENS = 6, 96, 160, 2, 75


@pytest.fixture(scope="module")
def M():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_scaled_amd as m
    return m


def normal(gen, *shape, std=1.0):
    import torch
    return (torch.randn(*shape, generator=gen) * std).to(torch.bfloat16)


def layer64(x, logits, w1, w2, b1, b2):
    """SwiGLU experts, weighted by the softmax of the TOPK logits."""
    import torch
    top = logits.topk(TOPK, dim=1)
    wt = torch.softmax(top.values, dim=1)
    y = torch.zeros_like(x)
    for j in range(TOPK):
        k = top.indices[:, j]
        pre = torch.matmul(w1[k], x[:, :, None])[:, :, 0] + b1[k]
        a = pre[:, :F] * torch.sigmoid(pre[:, :F]) * pre[:, F:]
        y = y + wt[:, j, None] * (torch.matmul(w2[k], a[:, :, None])[:, :, 0] + b2[k])
    return y


def rel(a, b):
    return ((a.double().cpu() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("captured", [False, True])
def test_trained_clipped_quantized_and_served(M, captured):
    import torch
    gen = torch.Generator().manual_seed(1)
    master = [torch.randn(E, 2 * F, H, generator=gen) * H ** -0.5, torch.randn(E, H, F, generator=gen) * F ** -0.5,
              torch.randn(E, 2 * F, generator=gen) * 0.1, torch.randn(E, H, generator=gen) * 0.1]
    master = [t.cuda() for t in master]
    names = ["dw1", "dw2", "db1", "db2"]
    params = [t.to(torch.bfloat16) for t in master]
    layer = M.MoELayer(M.GatedMLP("swiglu", *params), TOPK)
    x, dy = (normal(gen, TOKENS, H).cuda() for _ in range(2))
    logits = torch.randn(TOKENS, E, generator=gen).cuda()
    lr, limit = 0.05, 2.0

    def step():
        y = layer.forward(x, logits)
        g = layer.backward(dy)
        grads = [g[n] for n in names]
        clipped = [torch.empty_like(t) for t in grads]
        norm = M.clip_grad_norm(grads, limit, out=clipped)
        for w, p, c in zip(master, params, clipped):
            w.sub_(lr * c)
            p.copy_(w)
        return y, grads, clipped, norm

    run, outs = step, None
    if captured:
        layer.forward(x, logits)
        M.clip_grad_norm([t.clone() for t in layer.backward(dy).values()], limit)
        # (the capture itself runs nothing: the first replay is the first step)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            outs = step()

        def run():
            graph.replay()
            return outs

    for i in range(4):
        x.copy_(normal(gen, TOKENS, H))
        dy.copy_(normal(gen, TOKENS, H))
        logits.copy_(torch.randn(TOKENS, E, generator=gen))
        leaves = [p.double().cpu().requires_grad_() for p in params]
        before = [w.clone() for w in master]
        y, grads, clipped, norm = run()
        torch.cuda.synchronize()
        ref = layer64(x.double().cpu(), logits.double().cpu(), *leaves)
        # at most five roundings to BF16 between the inputs and any of these
        assert rel(y, ref.detach()) < math.sqrt(5) * UBF
        (ref * dy.double().cpu()).sum().backward()
        for n, g, leaf in zip(names, grads, leaves):
            assert g.dtype == torch.float32 and rel(g, leaf.grad) < math.sqrt(5) * UBF, (i, n)
        exact = norm64([g.cpu() for g in grads])
        assert exact > limit and abs(norm.item() - exact) <= 1.01 * 2.0 ** -24 * exact
        for g, c, w, b, p in zip(grads, clipped, master, before, params):
            want = g.double() * (limit / (exact + 1e-6))
            assert ((c.double() - want).abs() <= 3 * 2.0 ** -24 * want.abs() + 1e-44).all()
            assert torch.equal(w, b - lr * c) and torch.equal(p, w.to(torch.bfloat16))

    # served: the weights in 4 bits, in the same layer and in the formula
    codes = [M.w4_quantize(p, group=32, zeros=True) for p in params[:2]]
    served = M.MoELayer(M.W4GatedMLP("swiglu", *[M.w4_pack(*c) for c in codes], *params[2:]), TOPK)
    values = [values64(*[t.cpu() for t in c]) for c in codes]
    for tokens in (TOKENS, 1):
        y = served.forward(x[:tokens], logits[:tokens])
        ref = layer64(x[:tokens].double().cpu(), logits[:tokens].double().cpu(), *values, *[p.double().cpu() for p in params[2:]])
        assert rel(y, ref) < math.sqrt(4) * UBF
        # and no further from the trained layer than 4 bits take it: a step of 1/15 of a group's range, about 4 deviations
        # of its weights, leaves 4 / 15 / sqrt(12) = 0.077 of a weight's size, twice in a block of three products of them
        assert rel(y, layer.forward(x[:tokens], logits[:tokens]).double().cpu()) < 0.25


def test_two_streams_at_once(M):
    """Two blocks that train and a third that serves, each on a stream of its own at the same time: as one after the other."""
    import torch
    gen = torch.Generator().manual_seed(7)
    splits, h, f = [200, 0, 313], 256, 512
    m = sum(splits)
    w1, w2 = normal(gen, 3, 2 * f, h, std=h ** -0.5).cuda(), normal(gen, 3, h, f, std=f ** -0.5).cuda()
    q1, q2 = (M.w4_pack(*M.w4_quantize(w)) for w in (w1, w2))
    xs, dys = ([normal(gen, m, h).cuda() for _ in range(2)] for _ in range(2))
    p = torch.rand(m, generator=gen).cuda()

    def trained(i):
        mlp = M.GatedMLP("swiglu", w1, w2)
        out = []
        for _ in range(4):
            y = mlp.forward(xs[i], p, splits)
            g = mlp.backward(dys[i])
            out = [y, g["dx1"], g["dprobs"], M.clip_grad_norm([g["dw1"], g["dw2"]], 0.5), g["dw1"], g["dw2"]]
        return out

    def served(_):
        mlp = M.W4GatedMLP("swiglu", q1, q2)
        return [mlp.forward(xs[0], p, splits) for _ in range(8)]

    work = [(trained, 0), (trained, 1), (served, 0)]
    ref = [fn(i) for fn, i in work]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in work], []
    for (fn, i), s in zip(work, streams):
        with torch.cuda.stream(s):
            got.append(fn(i))
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_two_graphs_share_a_workspace(M):
    """Two captured clips of different gradients with one workspace, replayed in turn: each its own norm, every time."""
    import torch
    gen = torch.Generator().manual_seed(8)
    sizes = [[300000, 7], [5] * 150 + [2000000]]
    grads = [[torch.empty(n, device="cuda") for n in s] for s in sizes]
    outs = [[torch.empty_like(g) for g in gs] for gs in grads]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    run = lambda i: M.clip_grad_norm(grads[i], 1.0, out=outs[i], workspace=ws)
    for i in range(2):
        for g in grads[i]:
            g.normal_()
        run(i)
    torch.cuda.synchronize()
    graphs, norms = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            norms.append(run(i))
    for r in range(3):
        for i in range(2):
            for g in grads[i]:
                g.copy_(torch.randn(g.numel(), generator=gen) * (r + 1))
        for i in (0, 1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            exact = norm64([g.cpu() for g in grads[i]])
            assert abs(norms[i].item() - exact) <= 1.01 * 2.0 ** -24 * exact
            for g, o in zip(grads[i], outs[i]):
                want = g.double() / (exact + 1e-6)
                assert ((o.double() - want).abs() <= 3 * 2.0 ** -24 * want.abs() + 1e-44).all()
        assert torch.equal(run(0), norms[0])
