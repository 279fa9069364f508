"""MXFP4 (E2M1 elements, one E8M0 scale per 32) without a GPU: the oracle's rule against a search over
the element values and closed forms, the library's buffer sizes, and the refusals of its entry points."""

import itertools

import numpy as np
import pytest

from oracle import codecs
from oracle import gemm as G
from oracle import quant as Q
from tests.test_abi import FAKE, _expect, _fake_device_groups


def test_oracle_scale_codes_and_nearest_values():
    """The scale in closed form, and every element the nearest E2M1 multiple of it by search over all
    sixteen codes (a tie goes to the even code), saturated at 6."""
    rng = np.random.default_rng(0)
    x = np.float32(rng.standard_normal((64, 64)) * np.exp2(rng.integers(-20, 20, (64, 1)))).astype(np.float64)
    x[0], x[1, 32:] = 0.0, 0.0
    x[2, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.5]   # halfway points under scale 1, and past the end
    x[2, 8:32] = 0.0
    data, scales = Q.mxfp4_quantize_rows(x)
    codes = codecs.unpack_e2m1(data.reshape(64, 32))
    mags = codecs.E2M1_MAGS
    for r, b in itertools.product(range(64), range(2)):
        blk, c = x[r, 32 * b:32 * b + 32], int(scales[r, b])
        top = np.max(np.abs(blk))
        want = 0 if top == 0 else int(np.floor(np.log2(top))) - 2 + 127
        assert c == want, (r, b)
        v = np.minimum(np.abs(blk) / 2.0 ** (c - 127), 6.0)
        got = codecs.e2m1_decode(codes[r, 32 * b:32 * b + 32])
        assert np.array_equal(np.abs(np.abs(got) - v), np.min(np.abs(mags[None] - v[:, None]), axis=1)), (r, b)
        assert np.array_equal(np.signbit(got), np.signbit(blk))
    assert np.array_equal(codecs.e2m1_decode(codes[2, :8]), [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0])


def test_oracle_layouts_round_trip():
    """Codes and scales read back through the documented layouts give the quantized values, rowwise and
    columnwise (padding tokens are zeros)."""
    rng = np.random.default_rng(1)
    splits, w = [3, 0, 130, 61], 96
    x = rng.standard_normal((sum(splits), w)).astype(np.float32).astype(np.float64)
    q = Q.quantize_grouped(x, splits, "mxfp4")
    assert (len(q["row_data"]), len(q["row_scales"])) == Q.qtensor_nbytes("mxfp4", False, splits, w)
    assert (len(q["col_data"]), len(q["col_scales"])) == Q.qtensor_nbytes("mxfp4", True, splits, w)
    rows = G.dequant_row_grouped("mxfp4", q["row_data"], q["row_scales"], splits, w)
    cols = G.dequant_col_grouped("mxfp4", q["col_data"], q["col_scales"], splits, w)
    # scale 2^(e - 2) with 2^e <= amax < 2^(e + 1): off by at most 2 scales (saturation, 6 to 8)
    assert np.max(np.abs(rows - x)) <= np.exp2(np.floor(np.log2(np.max(np.abs(x)))) - 1)
    lo = 0
    for g, m in enumerate(splits):
        assert cols[g].shape == (w, -(-m // 128) * 128)
        assert not cols[g][:, m:].any()
        if m:
            assert np.corrcoef(cols[g][:, :m].ravel(), x[lo:lo + m].T.ravel())[0, 1] > 0.98
        lo += m


def test_buffer_sizes():
    from moe_grouped_scaled_amd import _native as N
    for splits in ([64, 128, 32, 32], [0, 1, 31, 33, 64], [1]):
        for col in (False, True):
            for w in (32, 96, 512):
                d, s = Q.qtensor_nbytes("mxfp4", col, splits, w)
                assert N.qtensor_nbytes("mxfp4", col, splits, w, "data") == d
                assert N.qtensor_nbytes("mxfp4", col, splits, w, "scales") == s
        assert N.qtensor_nbytes("mxfp4", False, splits, 96, "group_scale") == 0
    dg = _fake_device_groups(4, 300)
    assert N.qtensor_nbytes("mxfp4", True, dg, 96, "data") == 128 * (3 + 4) * 96 // 2
    assert N.qtensor_nbytes("mxfp4", False, dg, 96, "scales") == 4 * 300


def test_refusals():
    """Same checks as the other formats; no group scale or group amax is asked for; the Hadamard
    transform and the activation epilogue are other formats' recipes; scale arrays stay below 2 GiB."""
    import torch
    from moe_grouped_scaled_amd import _native as N
    act = N.act_params("srelu")
    q = N.QBuf(FAKE, FAKE, None)
    c, cb = torch.empty(1, dtype=torch.float32), torch.empty(1, dtype=torch.bfloat16)
    f, g = N.grouped_scaled_act_fwd, N.grouped_gemm_mx
    _expect(-2, f, act, "mxfp4", [32], 48, FAKE, FAKE, out_row=q, stream=0, match="multiple of 32")
    _expect(-1, f, act, "mxfp4", [32], 64, FAKE, FAKE, stream=0, match="no output")
    _expect(-1, f, act, "mxfp4", [32], 64, FAKE, FAKE, out_row=N.QBuf(FAKE, None, None), stream=0, match="scales")
    _expect(-3, f, act, "mxfp4", [32], 64, FAKE, FAKE, out_col=N.QBuf(FAKE, FAKE, None, N.RHT_ON), stream=0, match="NVFP4")
    _expect(-2, N.grouped_mx_quantize, "mxfp4", [65536], 32768, FAKE, out_row=q, stream=0, match="2\\^31")
    _expect(-2, g, "fprop", "mxfp4", [32, 32], 63, 64, 64, q, q, c, stream=0, match="split sum")
    _expect(-2, g, "fprop", "mxfp4", [32, 32], 64, 64, 48, q, q, c, stream=0, match="multiple of 32")
    _expect(-2, g, "fprop", "mxfp4", [32, 32], 64, 40, 64, q, q, c, stream=0, match="multiple of 32")
    _expect(-1, g, "wgrad", "mxfp4", [32], 64, 64, 32, q, q, c, bias=FAKE, stream=0, match="bias")
    _expect(-3, g, "fprop", "mxfp4", [32], 32, 64, 64, q, q, cb, accumulate=True, stream=0)
    _expect(-1, g, "fprop", "mxfp4", [32], 32, 64, 64, q, N.QBuf(FAKE, None, None), c, stream=0, match="operand B")
    _expect(-2, g, "fprop", "mxfp4", [32], 32, 1 << 24, 1 << 12, q, q, c, stream=0, match="2 GiB")
    with pytest.raises(AssertionError, match="NVFP4"):
        from moe_grouped_scaled_amd.expert_mlp import ExpertMLP
        w = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
        ExpertMLP("srelu", "mxfp4", w, w, rht_signs=1)
