"""`GatedMLP` with delayed weight gradients: none is lost, and none is computed from data that changed meanwhile."""

import pytest

from test_gpu_gated_mlp import layer_case, params

pytestmark = pytest.mark.gpu

SPLITS, H, F = [20, 0, 45], 72, 88


@pytest.fixture(scope="module")
def M():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_scaled_amd as m
    return m


def case(seed, bias=True):
    import torch
    dev = [None if t is None else t.cuda() for t in params(3, H, F, seed, bias)]
    gen = torch.Generator().manual_seed(seed + 1)
    rows = lambda: torch.randn(65, H, generator=gen).to(torch.bfloat16).cuda()
    return dev, [(rows(), rows(), torch.rand(65, generator=gen).cuda()) for _ in range(2)]


def steps(mlp, batch, delayed):
    x, dy, p = batch
    y = mlp.forward(x, p, SPLITS)
    g = mlp.backward(dy)
    if delayed:
        g.update(mlp.backward_dw())
    return dict(g, y=y)


def equal(a, b):
    import torch
    assert set(a) == set(b)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_a_second_backward_is_refused(M):
    """The first one's weight gradients are computed, then the second backward goes on from its own forward."""
    dev, (one, two) = case(60)
    now = M.GatedMLP("swiglu", *dev)
    want = [steps(now, b, False) for b in (one, two)]
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True)
    first = dict(y=mlp.forward(one[0], one[2], SPLITS))
    first.update(mlp.backward(one[1]))
    second = dict(y=mlp.forward(two[0], two[2], SPLITS))
    for _ in range(2):
        with pytest.raises(ValueError, match="still to be computed"):
            mlp.backward(two[1])
    first.update(mlp.backward_dw())
    second.update(mlp.backward(two[1]))
    second.update(mlp.backward_dw())
    equal(first, want[0])
    equal(second, want[1])


def test_dropped_weight_gradients(M):
    dev, (one, two) = case(62)
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True)
    mlp.forward(one[0], one[2], SPLITS)
    mlp.backward(one[1])
    mlp.pending_wgrad = None
    equal(steps(mlp, two, True), steps(M.GatedMLP("swiglu", *dev), two, False))


def test_frozen_weights_have_none_to_lose(M):
    dev, batches = case(64)
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True, grad_fc1=False, grad_fc2=False)
    for x, dy, p in batches:
        mlp.forward(x, p, SPLITS)
        assert set(mlp.backward(dy)) == {"dx1", "dprobs"}
    assert mlp.backward_dw() == {}


def test_layers_that_share_a_block(M):
    """A layer whose backward was refused can still go back once the weight gradients are computed."""
    import torch
    dev, x, logits, dy = layer_case(4, 64, 72, 19, 66, True)
    want = []
    for inp in (x, x.flip(0)):
        layer = M.MoELayer(M.GatedMLP("swiglu", *dev), 2)
        layer.forward(inp, logits)
        want.append(layer.backward(dy))
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True)
    a, b = M.MoELayer(mlp, 2), M.MoELayer(mlp, 2)
    a.forward(x, logits)
    first = a.backward(dy)
    b.forward(x.flip(0), logits)
    with pytest.raises(ValueError, match="still to be computed"):
        b.backward(dy)
    first.update(mlp.backward_dw())
    second = b.backward(dy)
    second.update(mlp.backward_dw())
    equal(first, want[0])
    equal(second, want[1])
    torch.cuda.synchronize()


def test_captured_in_two_graphs(M):
    """Forward and backward in one graph, the weight gradients in another, replayed for other inputs."""
    import torch
    dev, (one, two) = case(68)
    x, dy, p = [t.clone() for t in one]
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True)
    steps(mlp, (x, dy, p), True)
    torch.cuda.synchronize()
    a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        out = dict(y=mlp.forward(x, p, SPLITS))
        out.update(mlp.backward(dy))
    with torch.cuda.graph(b):
        out.update(mlp.backward_dw())
    for batch in (one, two, one):
        for t, s in zip((x, dy, p), batch):
            t.copy_(s)
        a.replay()
        b.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()}
        equal(got, steps(M.GatedMLP("swiglu", *dev), batch, False))


@pytest.mark.parametrize("delay", [False, True])
@pytest.mark.parametrize("name", ["x1", "probs"])
def test_a_change_after_the_forward_is_refused(M, name, delay):
    dev, (one, _) = case(70)
    x, dy, p = one
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=delay)
    mlp.forward(x, p, SPLITS)
    (x if name == "x1" else p).mul_(2)
    with pytest.raises(ValueError, match="%s was changed in place since the forward" % name):
        mlp.backward(dy)
    # a new forward takes it as it is now
    equal(steps(mlp, one, delay), steps(M.GatedMLP("swiglu", *dev), one, False))


@pytest.mark.parametrize("name,since", [("x1", "forward"), ("dy2", "backward")])
def test_a_change_before_delayed_gradients_is_refused(M, name, since):
    dev, (one, two) = case(72)
    x, dy, p = one
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True)
    mlp.forward(x, p, SPLITS)
    mlp.backward(dy)
    p.zero_()  # (nothing needs it any more)
    (x if name == "x1" else dy).copy_(two[0])
    for _ in range(2):
        with pytest.raises(ValueError, match="%s was changed in place since the %s" % (name, since)):
            mlp.backward_dw()


def test_what_no_gradient_needs_may_change(M):
    """x1 without FC1's gradients, dy2 without FC2's, both after a backward that was not delayed, parts of a buffer whose
    other parts change, and everything after a forward in inference mode."""
    import torch
    dev, (one, two) = case(74)
    x, dy, p = [t.clone() for t in one]
    want = steps(M.GatedMLP("swiglu", *dev), one, False)
    for off, var in (("grad_fc1", x), ("grad_fc2", dy)):
        mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True, **{off: False})
        mlp.forward(x, p, SPLITS)
        if off == "grad_fc1":
            x.zero_()
        g = mlp.backward(dy)
        if off == "grad_fc2":
            dy.zero_()
        g.update(mlp.backward_dw())
        for k in g:
            assert torch.equal(g[k], want[k]), k
        x, dy, p = [t.clone() for t in one]
    slots = torch.zeros((2, 65, H), dtype=torch.bfloat16, device="cuda")
    slots[0] = x
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True)
    got = dict(y=mlp.forward(slots[0], p, SPLITS))
    slots[1] = two[0]
    got.update(mlp.backward(dy))
    slots[1] = 0
    got.update(mlp.backward_dw())
    equal(got, want)
    with torch.inference_mode():
        xi = x.clone()
        assert torch.equal(mlp.forward(xi, p, SPLITS), want["y"])
        xi.zero_()


def test_graphs_whose_inputs_change_between_their_captures(M):
    import torch
    dev, (one, two) = case(76)
    x, dy, p = [t.clone() for t in one]
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True)
    steps(mlp, (x, dy, p), True)
    torch.cuda.synchronize()
    a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        out = dict(y=mlp.forward(x, p, SPLITS))
        out.update(mlp.backward(dy))
    for t, s in zip((x, dy, p), two):
        t.copy_(s)
    with torch.cuda.graph(b):
        out.update(mlp.backward_dw())
    for batch in (two, one, two):
        for t, s in zip((x, dy, p), batch):
            t.copy_(s)
        a.replay()
        b.replay()
        torch.cuda.synchronize()
        equal({k: v.clone() for k, v in out.items()}, steps(M.GatedMLP("swiglu", *dev), batch, False))
