"""MXFP4 weight gradients take the columnwise operands that the quantizing calls can write, no larger ones."""

import pytest

FAKE = 0x1000  # never dereferenced: the calls fail validation before any launch


@pytest.mark.parametrize("m,n", [(1 << 15, 32), (32, 1 << 15)])
def test_weight_gradient_operand_limit(m, n):
    import torch
    from moe_grouped_scaled_amd import _native as N
    q, c = N.QBuf(FAKE, FAKE, None), torch.empty(1)
    with pytest.raises(N.MgsError, match="2\\^31") as e:
        N.grouped_gemm_mx("wgrad", "mxfp4", [64, 1 << 16], m, n, 64 + (1 << 16), q, q, c, stream=0)
    assert e.value.code == -2
    with pytest.raises(N.MgsError, match="2\\^31"):
        N.grouped_mx_quantize("mxfp4", [64, 1 << 16], max(m, n), FAKE, out_col=q, stream=0)
