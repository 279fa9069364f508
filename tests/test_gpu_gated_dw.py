"""`GatedMLP.backward_dw` into given weight gradients: a call that is refused has added nothing, and can be made again."""

import pytest

from test_gpu_gated_delay import F, H, SPLITS, case, equal, steps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import moe_grouped_scaled_amd as m
    return m


def dw(name, dtype=None):
    import torch
    return torch.ones((3, 2 * F, H) if name == "dw1" else (3, H, F), dtype=dtype or torch.float32, device="cuda")


@pytest.mark.parametrize("name", ["dw1", "dw2"])
@pytest.mark.parametrize("wrong,match", [("none", "accumulate needs a"), ("bf16", "type"), ("shape", "shape"), ("strides", "contiguous"),
                                         ("offset", "16-byte"), ("cpu", "GPU")])
def test_a_refused_call_adds_nothing(M, name, wrong, match):
    import torch
    dev, (one, _) = case(80)
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True)
    want = steps(M.GatedMLP("swiglu", *dev), one, False)
    got = dict(y=mlp.forward(one[0], one[2], SPLITS))
    got.update(mlp.backward(one[1]))
    given = {n: dw(n) for n in ("dw1", "dw2")}
    t = given[name]
    bad = dict(given)
    bad[name] = {"none": lambda: None, "bf16": lambda: t.to(torch.bfloat16), "shape": lambda: t[:2], "cpu": lambda: t.cpu(),
                 "strides": lambda: t.transpose(1, 2).contiguous().transpose(1, 2),
                 "offset": lambda: torch.ones(t.numel() + 1, device="cuda")[1:].view(t.shape)}[wrong]()
    for _ in range(2):
        with pytest.raises(ValueError, match=match):
            mlp.backward_dw(**bad, accumulate=True)
    assert all((v == 1).all() for v in given.values())
    out = mlp.backward_dw(**given, accumulate=True)
    assert out["dw1"] is given["dw1"] and out["dw2"] is given["dw2"]
    for n in ("db1", "db2"):
        assert torch.equal(out[n], want[n])
    # one FP32 addition to the product's sum
    for n in ("dw1", "dw2"):
        assert torch.equal(given[n], want[n] + 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_given_gradients_are_written(M, dtype):
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    dev, (one, _) = case(82)
    want = steps(M.GatedMLP("swiglu", *dev, dw_dtype=dt), one, False)
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True)
    got = dict(y=mlp.forward(one[0], one[2], SPLITS))
    got.update(mlp.backward(one[1]))
    got.update(mlp.backward_dw(dw("dw1", dt), dw("dw2", dt)))
    equal(got, want)


@pytest.mark.parametrize("off", ["grad_fc1", "grad_fc2"])
def test_accumulate_needs_only_what_is_asked_for(M, off):
    import torch
    dev, (one, _) = case(84)
    want = steps(M.GatedMLP("swiglu", *dev), one, False)
    mlp = M.GatedMLP("swiglu", *dev, delay_wgrad=True, **{off: False})
    mlp.forward(one[0], one[2], SPLITS)
    mlp.backward(one[1])
    name = "dw2" if off == "grad_fc1" else "dw1"
    t = dw(name)
    assert set(mlp.backward_dw(**{name: t}, accumulate=True)) == {name, "db" + name[2]}
    assert torch.equal(t, want[name] + 1)
