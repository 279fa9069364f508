"""GPU parity of MXFP4: grouped quantization, the fused activations, the grouped products of every mode
and the expert-MLP step, against the float64 oracle.

Tolerances.  Codes and scales are bit-exact where the value before quantization is (identity, SReLU).
The GEMM gets the oracle's operand bytes: products of E2M1 values and powers of two are exact, so only
FP32 additions round.  An element is the sum of K / 32 block sums at most (in whatever order), each
addition off by at most one unit in the last place, 2^-23, of a partial sum, which never exceeds
S = sum |a b|: |error| <= (K / 32 + 8) 2^-23 S (8: the partial tiles, bias and accumulation), plus half a
step of the value, 2^-8 |c|, for a BF16 result.
"""

import numpy as np
import pytest

import workloads
from oracle import activations, codecs
from oracle import gemm as G
from oracle import mlp as M
from oracle import quant as Q
from tests.helpers import bf16_f64, bf16_host, compare_quantized, f32, rel_rms, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def N():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from moe_grouped_scaled_amd import _native
    return _native


def _elementwise(data, scales, rows, width):
    q = codecs.unpack_e2m1(np.asarray(data, np.uint8).reshape(rows, width // 2))
    s = np.repeat(codecs.e8m0_decode(Q.mx_scales_from_kstep(scales, rows, width)), 32, axis=1)
    return q, s, codecs.e2m1_decode(q) * s


def _dev_q(N, colwise, splits, width, q, guard=0):
    import torch
    t = N.QTensor("mxfp4", colwise, splits, width)
    pre = "col" if colwise else "row"
    t.data.copy_(torch.from_numpy(np.ascontiguousarray(q[pre + "_data"])))
    t.scales.copy_(torch.from_numpy(np.ascontiguousarray(q[pre + "_scales"])))
    return t


SPLITS = ([1], [64, 0, 37, 130], [0, 0, 5], [128, 256], [300, 1, 31, 33, 0, 96, 2])


@pytest.mark.parametrize("width", [32, 96, 160, 544])
@pytest.mark.parametrize("splits", SPLITS, ids=str)
def test_quantize_bit_exact(N, splits, width):
    """Row and column copies, column sums beside them; guard bytes behind every output stay."""
    import torch
    rng = np.random.default_rng(width + len(splits))
    m = sum(splits)
    bits = workloads.normal_bf16(rng, (m, width))
    x = bf16_f64(bits)
    if m > 2:
        bits[0] = 0                                        # a row of zeros
        bits[1, :32] = np.array([0x0001, 0x8001] * 16)     # BF16 subnormals
        bits[2, :32] = np.array([0x7F7F, 0xFF7F, 0x3F80, 0x0080] * 8)  # the largest beside small ones
        x = bf16_f64(bits)
    ref = Q.quantize_grouped(x, splits, "mxfp4")
    qr, qc = N.QTensor("mxfp4", False, splits, width), N.QTensor("mxfp4", True, splits, width)
    bufs = []
    for t in (qr, qc):
        for name in ("data", "scales"):
            n = getattr(t, name).numel()
            b = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
            bufs.append((b, n))
            setattr(t, name, b[:n])
    N.grouped_mx_quantize("mxfp4", splits, width, to_dev_bf16(bits), qr, qc)
    torch.cuda.synchronize()
    for t, pre in ((qr, "row"), (qc, "col")):
        assert np.array_equal(t.data.cpu().numpy(), ref[pre + "_data"]), pre
        assert np.array_equal(t.scales.cpu().numpy(), ref[pre + "_scales"]), pre
    for b, n in bufs:
        assert bool((b[n:] == 0xA5).all())


@pytest.mark.parametrize("kind", ["srelu", "tanh_srelu", "gelu", "swiglu", "clamped_swiglu"])
def test_act_forward_and_backward(N, kind):
    import torch
    splits = [64, 0, 37, 130]
    wa = 160
    d = workloads.act_case(kind, splits, 2 * wa if kind in ("swiglu", "clamped_swiglu") else wa, seed=7, std=1.5)
    m, w_in = int(d["splits"].sum()), d["width_in"]
    act = N.act_params(kind)
    par = {"s": 2.0} if kind == "tanh_srelu" else {"limit": 7.0} if kind == "clamped_swiglu" else {}
    x64, p64, dy64 = bf16_f64(d["x"]), d["p"].astype(np.float64), bf16_f64(d["dy"])
    x, p, dy = to_dev_bf16(d["x"]), to_dev(d["p"]), to_dev_bf16(d["dy"])
    y = activations.scaled_act_fwd(kind, x64, p64, **par)
    dx64, dp64 = activations.scaled_act_bwd(kind, x64, dy64, p64, **par)
    row, col = N.QTensor("mxfp4", False, splits, wa), N.QTensor("mxfp4", True, splits, wa)
    N.grouped_scaled_act_fwd(act, "mxfp4", splits, w_in, x, p, row, col)
    frow, frow_bf = N.QTensor("mxfp4", False, splits, wa), torch.empty((m, w_in), dtype=torch.bfloat16, device="cuda")
    N.grouped_scaled_act_fwd_f32(act, "mxfp4", splits, w_in, x.float(), p, frow, None, x_bf16_out=frow_bf)
    dxr, dxc = N.QTensor("mxfp4", False, splits, w_in), N.QTensor("mxfp4", True, splits, w_in)
    again = N.QTensor("mxfp4", True, splits, wa)
    dense, dp = torch.empty((m, w_in), dtype=torch.bfloat16, device="cuda"), torch.empty(m, device="cuda")
    N.grouped_scaled_act_bwd(act, "mxfp4", splits, w_in, x, dy, p, dx=dense, dx_row=dxr, dx_col=dxc, dprobs=dp, act_col=again)
    torch.cuda.synchronize()
    exact = kind == "srelu"
    for what, got, ref64, width in (("y", (row, col), y, wa), ("dx", (dxr, dxc), dx64, w_in)):
        ref = Q.quantize_grouped(ref64, splits, "mxfp4")
        if exact:
            assert np.array_equal(got[0].data.cpu().numpy(), ref["row_data"]), what
            assert np.array_equal(got[1].data.cpu().numpy(), ref["col_data"]), what
            assert np.array_equal(got[0].scales.cpu().numpy(), ref["row_scales"]), what
            assert np.array_equal(got[1].scales.cpu().numpy(), ref["col_scales"]), what
            continue
        # FP32 activations differ from the oracle's in the last bits: an element next to a rounding
        # border moves one step of the grid (at most one in a thousand: the borders are ~2^-20 wide
        # against steps of 2^-2)
        compare_quantized("mxfp4", _elementwise(got[0].data.cpu(), got[0].scales.cpu(), m, width),
                          _elementwise(ref["row_data"], ref["row_scales"], m, width))
        coff = Q.col_offsets(splits)
        for g in range(len(splits)):
            mp = int(coff[g + 1] - coff[g])
            if mp == 0:
                continue
            cut = lambda a, div: np.asarray(a)[width * int(coff[g]) // div:width * int(coff[g + 1]) // div]
            compare_quantized("mxfp4", _elementwise(cut(got[1].data.cpu(), 2), cut(got[1].scales.cpu(), 32), width, mp),
                              _elementwise(cut(ref["col_data"], 2), cut(ref["col_scales"], 32), width, mp))
    # regenerated and FP32-input copies: the same bits as the forward's
    assert torch.equal(again.data, col.data) and torch.equal(again.scales, col.scales)
    assert torch.equal(frow.data, row.data) and torch.equal(frow.scales, row.scales) and torch.equal(frow_bf, x)
    # dprobs: a sum of wa products in FP32, plus the activation's own few roundings
    a64 = activations.scaled_act_fwd(kind, x64, np.ones(m), **par)
    bound = (wa + 16) * 2.0 ** -23 * np.sum(np.abs(dy64 * a64), axis=1) + 1e-30
    assert np.all(np.abs(f32(dp) - dp64) <= bound)


def _bound(absolute, k, c=None):
    b = (k / 32 + 8) * 2.0 ** -23 * absolute
    return b if c is None else b + 2.0 ** -8 * np.abs(c)


def _operands(seed, splits, n, k, fmt_mode):
    rng = np.random.default_rng(seed)
    e, m = len(splits), sum(splits)
    x = bf16_f64(workloads.normal_bf16(rng, (m, k)))
    w = bf16_f64(workloads.normal_bf16(rng, (e, n, k) if fmt_mode != "dgrad" else (e, k, n), 0.02))
    return rng, x, w


SHAPES = [([1], 32, 32), ([1, 0, 2], 64, 96), ([5], 256, 4096), ([16, 3, 0, 17], 160, 544), ([33, 64, 65], 288, 256),
          ([0, 100, 37, 256], 160, 544), ([300, 257], 512, 384), ([513], 96, 1120)]


@pytest.mark.parametrize("device_splits", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("mode", ["fprop", "dgrad"])
@pytest.mark.parametrize("splits,n,k", SHAPES, ids=str)
def test_fprop_dgrad(N, splits, n, k, mode, out, device_splits):
    import torch
    e, m = len(splits), sum(splits)
    rng, x, w = _operands(n + k, splits, n, k, mode)
    bias = workloads.normal_bf16(rng, (e, n), 0.5)
    qx = Q.quantize_grouped(x, splits, "mxfp4", colwise=False)
    a64 = G.dequant_row_grouped("mxfp4", qx["row_data"], qx["row_scales"], splits, k)
    if mode == "fprop":
        qw = Q.quantize_grouped(w.reshape(e * n, k), [n] * e, "mxfp4", colwise=False)
        b64 = list(G.dequant_row_grouped("mxfp4", qw["row_data"], qw["row_scales"], [n] * e, k).reshape(e, n, k))
        B = _dev_q(N, False, [n] * e, k, qw)
    else:
        qw = Q.quantize_grouped(w.reshape(e * k, n), [k] * e, "mxfp4", rowwise=False)
        b64 = G.dgrad_weight(G.dequant_col_grouped("mxfp4", qw["col_data"], qw["col_scales"], [k] * e, n), k)
        B = _dev_q(N, True, [k] * e, n, qw)
    ref = G.gemm_grouped_m(a64, b64, splits, bias=bf16_f64(bias))
    size = G.gemm_grouped_m(np.abs(a64), [np.abs(b) for b in b64], splits, bias=np.abs(bf16_f64(bias)))
    dt = torch.float32 if out == "f32" else torch.bfloat16
    print("case:", mode, splits, n, k, out, device_splits, flush=True)
    if device_splits:
        cap = m + 37
        dg = N.DeviceGroups(e, cap)
        dg.splits.copy_(torch.tensor(splits))
        dg.update()
        A = N.QTensor("mxfp4", False, dg, k)
        A.data.fill_(0xFF)
        A.scales.fill_(0xFF)                     # bytes past the rows in use are no numbers
        A.data[:m * k // 2].copy_(torch.from_numpy(qx["row_data"]))
        A.scales.view(-(-k // 128), cap, 4)[:, :m].copy_(torch.from_numpy(qx["row_scales"].reshape(-1, m, 4)))
        c = torch.full((cap, n), 7.0, dtype=dt, device="cuda")
        N.grouped_gemm_mx(mode, "mxfp4", dg, cap, n, k, A, B, c, bias=to_dev_bf16(bias))
        torch.cuda.synchronize()
        assert bool((c[m:] == 7.0).all())        # rows behind the last group's stay
        c = c[:m]
    else:
        A = _dev_q(N, False, splits, k, qx)
        c = torch.full((m, n), float("nan"), dtype=dt, device="cuda")
        N.grouped_gemm_mx(mode, "mxfp4", splits, m, n, k, A, B, c, bias=to_dev_bf16(bias))
        torch.cuda.synchronize()
    got = f32(c) if out == "f32" else bf16_f64(bf16_host(c))
    assert np.all(np.abs(got - ref) <= _bound(size, k, None if out == "f32" else ref))


@pytest.mark.parametrize("device_splits", [False, True])
@pytest.mark.parametrize("out,accumulate", [("f32", False), ("f32", True), ("bf16", False)])
@pytest.mark.parametrize("splits,mw,n", [([1], 32, 64), ([0, 100, 37, 256], 160, 288), ([300, 0, 513], 512, 96)], ids=str)
def test_wgrad(N, splits, mw, n, out, accumulate, device_splits):
    import torch
    rng = np.random.default_rng(mw + n)
    e, m = len(splits), sum(splits)
    dy, x = bf16_f64(workloads.normal_bf16(rng, (m, mw))), bf16_f64(workloads.normal_bf16(rng, (m, n)))
    qa, qb = Q.quantize_grouped(dy, splits, "mxfp4", rowwise=False), Q.quantize_grouped(x, splits, "mxfp4", rowwise=False)
    a64 = G.dequant_col_grouped("mxfp4", qa["col_data"], qa["col_scales"], splits, mw)
    b64 = G.dequant_col_grouped("mxfp4", qb["col_data"], qb["col_scales"], splits, n)
    ref = G.gemm_grouped_k(a64, b64)
    size = G.gemm_grouped_k([np.abs(a) for a in a64], [np.abs(b) for b in b64])
    old = rng.standard_normal((e, mw, n)).astype(np.float32)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    c = to_dev(old).to(dt)
    if accumulate:
        ref, size = ref + old, size + np.abs(old)
    print("case:", splits, mw, n, out, accumulate, device_splits, flush=True)
    if device_splits:
        cap = m + 200
        dg = N.DeviceGroups(e, cap)
        dg.splits.copy_(torch.tensor(splits))
        dg.update()
        ops = []
        for q, w in ((qa, mw), (qb, n)):
            t = N.QTensor("mxfp4", True, dg, w)
            t.data.fill_(0xFF)
            t.scales.fill_(0xFF)
            t.data[:len(q["col_data"])].copy_(torch.from_numpy(q["col_data"]))
            t.scales[:len(q["col_scales"])].copy_(torch.from_numpy(q["col_scales"]))
            ops.append(t)
        N.grouped_gemm_mx("wgrad", "mxfp4", dg, mw, n, cap, *ops, c, accumulate=accumulate)
    else:
        N.grouped_gemm_mx("wgrad", "mxfp4", splits, mw, n, m, _dev_q(N, True, splits, mw, qa), _dev_q(N, True, splits, n, qb), c,
                          accumulate=accumulate)
    torch.cuda.synchronize()
    got = f32(c) if out == "f32" else bf16_f64(bf16_host(c.view(e * mw, n))).reshape(e, mw, n)
    assert np.all(np.abs(got - ref) <= _bound(size, max(splits) + 128, None if out == "f32" else ref))


@pytest.mark.parametrize("scale", [0, 1, 60, 127, 190, 247])
def test_scales_over_the_whole_range(N, scale):
    """Operand scales far from 1 multiply out as powers of two: the same integers, shifted exactly."""
    import torch
    rng = np.random.default_rng(scale)
    m, n, k = 40, 64, 160
    a, b = rng.integers(0, 16, (m, k)).astype(np.uint8), rng.integers(0, 16, (n, k)).astype(np.uint8)
    other = 254 - scale
    qa = {"row_data": codecs.pack_e2m1(a).reshape(-1), "row_scales": Q.mx_scales_to_kstep(np.full((m, k // 32), scale, np.uint8))}
    qb = {"row_data": codecs.pack_e2m1(b).reshape(-1), "row_scales": Q.mx_scales_to_kstep(np.full((n, k // 32), other, np.uint8))}
    c = torch.empty((m, n), device="cuda")
    N.grouped_gemm_mx("fprop", "mxfp4", [m], m, n, k, _dev_q(N, False, [m], k, qa), _dev_q(N, False, [n], k, qb), c)
    torch.cuda.synchronize()
    assert np.array_equal(f32(c), codecs.e2m1_decode(a) @ codecs.e2m1_decode(b).T)


@pytest.mark.parametrize("kind,recompute", [("srelu", False), ("srelu", True), ("swiglu", True)])
def test_expert_mlp_step(N, kind, recompute):
    """The whole step in this recipe against the oracle step.  The chained quantities see rare moves of
    one grid step (a BF16 rounding apart before quantization): each is half the widest relative step,
    1/6 to 1/3 of a value, in far fewer than one element in a hundred, so 2 % of the tensor's RMS."""
    import torch
    from moe_grouped_scaled_amd.expert_mlp import ExpertMLP
    e, splits, h, f = 4, [64, 0, 96, 37], 128, 128
    rng = np.random.default_rng(3)
    f_in = 2 * f if kind == "swiglu" else f
    m = sum(splits)
    x1, w1 = workloads.normal_bf16(rng, (m, h)), workloads.normal_bf16(rng, (e, f_in, h), 0.05)
    w2, b1 = workloads.normal_bf16(rng, (e, h, f), 0.05), workloads.normal_bf16(rng, (e, f_in), 0.05)
    b2, p, dy2 = workloads.normal_bf16(rng, (e, h), 0.05), workloads.uniform_f32(rng, m), workloads.normal_bf16(rng, (m, h))
    mlp = ExpertMLP(kind, "mxfp4", to_dev_bf16(w1), to_dev_bf16(w2), to_dev_bf16(b1), to_dev_bf16(b2), recompute=recompute)
    y2 = mlp.forward(to_dev_bf16(x1), to_dev(p), splits)
    g = mlp.backward(to_dev_bf16(dy2))
    torch.cuda.synchronize()
    ref = M.mlp_step(kind, "mxfp4", splits, *[bf16_f64(t) for t in (x1, w1, b1, w2, b2)], p.astype(np.float64), bf16_f64(dy2),
                     recompute=recompute)
    got = {"y2": bf16_f64(bf16_host(y2)), "dx1": bf16_f64(bf16_host(g["dx1"])), "dp": f32(g["dprobs"])}
    got.update({k: f32(g[k]) for k in ("dw1", "dw2", "db1", "db2")})
    for k, v in got.items():
        print(k, rel_rms(v, ref[k]), flush=True)
        assert rel_rms(v, ref[k]) <= 0.02, k
