"""Refusals of the BF16 products and the gated block: host checks, before anything touches a GPU."""

import pytest

FAKE = 0x10000  # never dereferenced: every call below fails validation before any launch


def _call(name, *args):
    from moe_grouped_scaled_amd import _native as N
    # (the groups stay alive in `args` until the call is over)
    rc = getattr(N.LIB, name)(*[a.ref if isinstance(a, N._GroupsArg) else a for a in args])
    return rc, N.last_error()


def _groups(splits):
    from moe_grouped_scaled_amd import _native as N
    return N._GroupsArg(splits)


def gemm(mode=0, splits=(4,), m=4, n=64, k=64, a=FAKE, b=FAKE << 4, c=FAKE << 8, dtype=0, bias=None, acc=0):
    return _call("mgs_grouped_gemm_bf16", mode, _groups(list(splits)), m, n, k, a, b, c, dtype, bias, acc, 0)


@pytest.mark.parametrize("change,code,match", [
    (dict(mode=3), -1, "unknown GEMM mode"), (dict(dtype=2), -1, "output dtype"), (dict(acc=1), -3, "FP32"),
    (dict(n=60), -2, "multiple of 8"), (dict(k=0), -2, "multiple of 8"), (dict(k=(1 << 20) + 8), -2, "above"),
    (dict(m=5), -2, "split sum"), (dict(mode=2, m=64, k=5), -2, "split sum"), (dict(mode=2, m=12, k=4), -2, "multiple of 8"),
    (dict(mode=2, m=64, k=4, bias=FAKE << 12), -1, "bias"), (dict(splits=(-1, 5)), -2, "negative"),
    (dict(splits=()), -1, "num_groups"), (dict(a=None), -1, "operand a"), (dict(b=None), -1, "operand b"),
    (dict(c=None), -1, "c is NULL"), (dict(mode=2, m=64, k=4, c=None), -1, "c is NULL"), (dict(a=FAKE + 8), -1, "a must be 16-byte"),
    (dict(bias=(FAKE << 12) + 2), -1, "bias must be 16-byte"), (dict(c=FAKE), -1, "c must not be or overlap a"),
    (dict(c=(FAKE << 4) + 16), -1, "c must not be or overlap b"), (dict(c=FAKE + 496), -1, "overlap a"),
    (dict(bias=(FAKE << 8) + 256), -1, "overlap bias"),
])
def test_gemm_refusals(change, code, match):
    rc, msg = gemm(**change)
    assert rc == code and match in msg, (rc, msg)


def test_gemm_without_rows():
    assert gemm(splits=(0, 0), m=0, a=None, b=None, c=None)[0] == 0


def fwd(kind="swiglu", splits=(4,), f=64, k=64, x=FAKE, w=FAKE << 4, bias=None, probs=None, h=FAKE << 8, pre=None, pdt=1, **kw):
    import ctypes
    from moe_grouped_scaled_amd import _native as N
    act = None if kind is None else ctypes.byref(N.act_params(kind, **kw))
    return _call("mgs_grouped_gated_fwd", act, _groups(list(splits)), f, k, x, w, bias, probs, h, pre, pdt, 0)


@pytest.mark.parametrize("change,code,match", [
    (dict(kind=None), -1, "act is NULL"), (dict(kind="gelu"), -1, "not a gated"), (dict(kind="clamped_swiglu", limit=0.0), -1, "limit"),
    (dict(kind="clamped_swiglu", alpha=float("nan")), -1, "finite"), (dict(f=4), -2, "multiple of 8"), (dict(k=9), -2, "multiple of 8"),
    (dict(x=None), -1, "x, w or h"), (dict(w=None), -1, "x, w or h"), (dict(h=None), -1, "x, w or h"),
    (dict(x=FAKE + 2), -1, "x must be 16-byte"), (dict(probs=FAKE + 2), -1, "probs must be 4-byte"),
    (dict(pre=FAKE << 8), -1, "overlap pre"), (dict(pre=FAKE + 256), -1, "overlap x"), (dict(probs=(FAKE << 8) + 508), -1, "overlap probs"),
    (dict(pre=FAKE << 9, pdt=2), -1, "type of pre"), (dict(pre=FAKE - 1040, pdt=1), -1, "overlap x"),
])
def test_gated_forward_refusals(change, code, match):
    rc, msg = fwd(**change)
    assert rc == code and match in msg, (rc, msg)


def bwd(kind="swiglu", splits=(4,), f=64, n=64, dy=FAKE, w2=FAKE << 4, pre=FAKE << 8, probs=None, dpre=FAKE << 12, h=None, dp=None,
        ws=None, wb=0, pdt=0):
    import ctypes
    from moe_grouped_scaled_amd import _native as N
    return _call("mgs_grouped_gated_bwd", ctypes.byref(N.act_params(kind)), _groups(list(splits)), f, n, dy, w2, pre, pdt, probs,
                 dpre, h, dp, ws, wb, 0)


@pytest.mark.parametrize("change,code,match", [
    (dict(kind="srelu"), -1, "not a gated"), (dict(f=65), -2, "multiple of 8"), (dict(n=-8), -2, "multiple of 8"),
    (dict(pre=None), -1, "dpre is NULL"), (dict(dpre=None), -1, "dpre is NULL"), (dict(dp=FAKE << 2), -1, "workspace of 32 bytes"),
    (dict(dp=FAKE << 2, ws=FAKE << 3, wb=31), -1, "got 31"), (dict(dpre=FAKE << 8), -1, "overlap pre"),
    (dict(h=(FAKE << 12) + 1008), -1, "dpre must not be or overlap h"), (dict(dp=FAKE << 2, ws=FAKE << 2, wb=32), -1, "overlap the workspace"),
    (dict(pdt=3), -1, "type of pre"), (dict(dpre=(FAKE << 8) + 1024, pdt=1), -1, "overlap pre"),
])
def test_gated_backward_refusals(change, code, match):
    rc, msg = bwd(**change)
    assert rc == code and match in msg, (rc, msg)


def test_workspace_bytes():
    from moe_grouped_scaled_amd import MgsError, grouped_gated_bwd_workspace_bytes as wb
    assert wb([3, 4], 64) == 4 * 7 * 2 and wb([3, 4], 72) == 4 * 7 * 4 and wb([0], 64) == 0
    with pytest.raises(MgsError, match="multiple of 8"):
        wb([3], 12)


def test_python_refusals():
    """What the Python functions check themselves, on CPU tensors."""
    import torch
    import moe_grouped_scaled_amd as m
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    for fn, match in [
        (lambda: m.grouped_gemm_bf16("up", [1], z(1, 8), z(1, 8, 8)), "mode"),
        (lambda: m.grouped_gemm_bf16("fprop", [1], z(1, 8), z(1, 8, 8)), "GPU"),
        (lambda: m.grouped_gemm_bf16("fprop", [1], torch.zeros(1, 8), z(1, 8, 8)), "type"),
        (lambda: m.grouped_gemm_bf16("fprop", [1], z(8), z(1, 8, 8)), "dimensions"),
        (lambda: m.grouped_gemm_bf16("fprop", [1], z(2, 16)[:, ::2], z(1, 8, 8)), "contiguous"),
        (lambda: m.grouped_gemm_bf16("fprop", [1], z(1, 8), z(1, 8, 8), accumulate=True), "accumulate"),
        (lambda: m.grouped_gemm_bf16("fprop", [1], z(1, 8), z(1, 8, 8), out_dtype=torch.float16), "out_dtype"),
        (lambda: m.grouped_gated_fwd("gelu", [1], z(1, 8), z(1, 16, 8)), "act must be"),
        (lambda: m.grouped_gated_bwd(3, [1], z(1, 8), z(1, 8, 8), z(1, 16)), "act must be"),
        (lambda: m.GatedMLP("srelu", z(1, 16, 8), z(1, 8, 8)), "kind"),
        (lambda: m.GatedMLP("glu", z(1, 16, 8), z(1, 8, 8), dw_dtype=torch.float16), "dw_dtype"),
    ]:
        with pytest.raises(ValueError, match=match):
            fn()
