"""Refusals of the 4-bit products and of the gradients' norm: host checks, before anything touches a GPU."""

import ctypes

import pytest

from test_gated_arguments import FAKE, _call, _groups


def test_nbytes():
    from moe_grouped_scaled_amd import _native as N
    f = N.LIB.mgs_w4_nbytes
    assert f(1, 16, 128, 128, 1) == 1024 + 64 and f(1, 16, 128, 128, 0) == 1024 + 32
    assert f(3, 17, 160, 32, 1) == 3 * 2 * 2 * (1024 + 256) and f(1, 1, 64, 64, 0) == 1024 + 64


@pytest.mark.parametrize("args,code,match", [
    ((0, 16, 128, 128), -1, "num_experts"), ((257, 16, 128, 128), -1, "num_experts"), ((1, 0, 128, 128), -2, "n = 0"),
    ((1, 16, 96, 64), -2, "multiple of the group"), ((1, 16, 0, 64), -2, "multiple of the group"), ((1, 16, 128, 16), -1, "group 16"),
    ((1, 16, (1 << 20) + 128, 128), -2, "above"), ((1, (1 << 20) + 1, 128, 128), -2, "outside"),
])
def test_shapes(args, code, match):
    rc, msg = _call("mgs_w4_nbytes", *args, 1)
    assert rc == code and match in msg
    rc, msg = _call("mgs_w4_pack", *args, FAKE, FAKE, FAKE, FAKE, 0)
    assert rc == code and match in msg
    rc, msg = _call("mgs_w4_quantize", *args, FAKE, FAKE, FAKE, FAKE, 0)
    assert rc == code and match in msg


def test_pack_and_quantize():
    good = (1, 16, 128, 64)
    for args, match in [((None, FAKE << 4, None, FAKE << 8), "NULL"), ((FAKE, FAKE << 4, None, FAKE), "overlap codes"),
                        ((FAKE, FAKE << 4, FAKE << 8, (FAKE << 8) - 16), "overlap zeros"), ((FAKE, (FAKE << 4) + 1, None, FAKE << 8), "scales must be"),
                        ((FAKE, FAKE << 4, None, (FAKE << 8) + 8), "out must be")]:
        rc, msg = _call("mgs_w4_pack", *good, *args, 0)
        assert rc == -1 and match in msg, msg
    for args, match in [((FAKE, None, FAKE << 4, None), "NULL"), ((FAKE + 8, FAKE << 4, FAKE << 8, None), "w must be"),
                        ((FAKE, FAKE + 4092, FAKE << 8, None), "overlap w"), ((FAKE, FAKE << 4, FAKE << 4, None), "overlap scales")]:
        rc, msg = _call("mgs_w4_quantize", *good, *args, 0)
        assert rc == -1 and match in msg, msg


def gemm(splits=(4,), n=64, k=64, group=64, zeros=1, x=FAKE, w=FAKE << 4, bias=None, c=FAKE << 8, dtype=0):
    return _call("mgs_grouped_gemm_w4", _groups(list(splits)), n, k, group, zeros, x, w, bias, c, dtype, 0)


def gated(kind="swiglu", splits=(4,), f=32, k=64, group=64, zeros=1, x=FAKE, w=FAKE << 4, bias=None, probs=None, h=FAKE << 8, **kw):
    from moe_grouped_scaled_amd import _native as N
    return _call("mgs_grouped_gated_w4", ctypes.byref(N.act_params(kind, **kw)), _groups(list(splits)), f, k, group, zeros, x, w,
                 bias, probs, h, 0)


@pytest.mark.parametrize("change,code,match", [
    (dict(dtype=3), -1, "output dtype"), (dict(splits=(-1,)), -2, "negative"), (dict(group=0), -1, "group 0"),
    (dict(k=96), -2, "multiple of the group"), (dict(x=None), -1, "NULL"), (dict(w=None), -1, "NULL"), (dict(c=None), -1, "NULL"),
    (dict(w=FAKE + 8), -1, "w must be"), (dict(c=FAKE + 510), -1, "overlap x"), (dict(c=(FAKE << 4) + 16), -1, "overlap w"),
    (dict(dtype=1, c=(FAKE << 8) + 2), -1, "c must be 4-byte"),
])
def test_gemm(change, code, match):
    rc, msg = gemm(**change)
    assert rc == code and match in msg, (rc, msg)


@pytest.mark.parametrize("change,code,match", [
    (dict(kind="gelu"), -1, "not a gated"), (dict(f=24), -2, "multiple of 16"), (dict(f=0), -2, "multiple of 16"),
    (dict(kind="clamped_swiglu", limit=-1.0), -1, "limit"), (dict(probs=FAKE + 2), -1, "probs must be"), (dict(h=FAKE), -1, "overlap x"),
    (dict(h=None), -1, "NULL"),
])
def test_gated(change, code, match):
    rc, msg = gated(**change)
    assert rc == code and match in msg, (rc, msg)


def test_no_rows():
    assert gemm(splits=(0, 0), x=None, w=None, c=None)[0] == 0
    assert gated(splits=(0,), x=None, w=None, h=None)[0] == 0


def grads(*rows):
    from moe_grouped_scaled_amd import _native as N
    t = (N.Grad * max(len(rows), 1))()
    for e, r in zip(t, rows):
        e.grad, e.out, e.numel, e.grad_dtype, e.out_dtype = r
    return t


@pytest.mark.parametrize("rows,kw,match", [
    ([(FAKE, FAKE, -1, 0, 0)], {}, "numel is negative"), ([(None, FAKE, 4, 0, 0)], {}, "grad is NULL"), ([(FAKE, FAKE, 4, 5, 0)], {}, "unknown dtype"),
    ([(FAKE + 1, FAKE, 4, 0, 0)], {}, "not aligned"), ([(FAKE, FAKE + 2, 4, 0, 1)], {}, "not aligned"),
    ([(FAKE, None, 4, 0, 0)], {}, "out is NULL"), ([(FAKE, FAKE, 4, 0, 0)], dict(norm=None), "norm is NULL"),
    ([(FAKE, FAKE, 4, 0, 0)], dict(wb=15), "workspace of 16"), ([(FAKE, FAKE, 4, 0, 0)], dict(ws=None), "workspace of 16"),
    ([(FAKE, FAKE, 4, 0, 0)], dict(max_norm=-1.0), "max_norm"), ([(FAKE, FAKE, 4, 0, 0)], dict(max_norm=float("inf")), "max_norm"),
    ([(FAKE, FAKE, 4, 0, 0)], dict(eps=float("nan")), "eps"), ([(FAKE, FAKE, 4, 0, 0)] * 2, dict(wb=24), "overlap"),
    ([(FAKE, FAKE, 4, 1, 0)], {}, "overlap"), ([(FAKE, FAKE + 8, 4, 0, 0), (FAKE + 14, FAKE + 14, 4, 0, 0)], dict(wb=24), "overlap"),
    ([(FAKE, FAKE, 4, 0, 0)], dict(norm=FAKE + 4), "overlap"), ([(FAKE, FAKE, 4, 0, 0)], dict(norm=FAKE << 4), "overlap"),
])
def test_norm(rows, kw, match):
    a = dict(norm=FAKE << 8, ws=FAKE << 4, wb=16, max_norm=1.0, eps=0.0)
    a.update(kw)
    rc, msg = _call("mgs_grad_norm", len(rows), grads(*rows), a["norm"], a["ws"], a["wb"], 1, a["max_norm"], a["eps"], 0)
    assert rc < 0 and match in msg, (rc, msg)


def test_norm_workspace():
    assert _call("mgs_grad_norm_workspace_bytes", 3, grads((FAKE, None, 2049, 0, 0), (None, None, 0, 1, 1), (FAKE, None, 1, 1, 1)))[0] == 32
    assert _call("mgs_grad_norm_workspace_bytes", 0, None)[0] == 8
    rc, msg = _call("mgs_grad_norm_workspace_bytes", -1, None)
    assert rc < 0 and "negative" in msg


def test_python_refusals():
    import torch
    import moe_grouped_scaled_amd as m
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    for fn, match in [
        (lambda: m.w4_pack(bf(1, 8, 8), bf(1, 8, 1)), "type"), (lambda: m.w4_pack(u8(8, 8), bf(1, 8, 1)), "dimensions"),
        (lambda: m.w4_pack(u8(1, 8, 16), bf(1, 8, 1)), "GPU"), (lambda: m.w4_quantize(bf(1, 8, 32)), "GPU"),
        (lambda: m.grouped_gemm_w4([1], bf(1, 8), 3, out_dtype=torch.float16), "out_dtype"),
        (lambda: m.W4GatedMLP("swiglu", 1, 2), "W4Tensor"), (lambda: m.W4GatedMLP("gelu", 1, 2), "kind"),
        (lambda: m.grad_norm([]), "empty"), (lambda: m.grad_norm([bf(3)]), "GPU"), (lambda: m.clip_grad_norm([bf(3)], 1.0, out=[]), "out has"),
    ]:
        with pytest.raises(ValueError, match=match):
            fn()


def test_packed_weights_have_their_size():
    """A W4Tensor around other data would let the products read past its end; 32-bit arguments are not cut off."""
    import torch
    import moe_grouped_scaled_amd as m
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)
    size = m._native.LIB.mgs_w4_nbytes(2, 40, 96, 32, 1)
    t = m.W4Tensor(u8(size), (2, 40, 96), 32, True)
    assert t.nbytes() == size and t.shape == (2, 40, 96)
    for data in (u8(size - 1), u8(size + 16), u8(size).view(torch.int8), u8(2 * size)[::2], 3):
        with pytest.raises(ValueError, match="%d bytes" % size):
            m.W4Tensor(data, (2, 40, 96), 32, True)
    with pytest.raises(m.MgsError, match="not 32, 64 or 128"):
        m.W4Tensor(u8(size), (2, 40, 96), 48, True)
    for fn in (lambda: m.W4Tensor(u8(size), (2, 40, 96), 2 ** 32 + 32, True), lambda: m.w4_quantize(u8(4), group=2 ** 32 + 32),
               lambda: m.w4_quantize(u8(4), group=-32), lambda: m.W4Tensor(u8(size), (2 ** 32 + 2, 40, 96), 32, True)):
        with pytest.raises(ValueError, match="out of range"):
            fn()
