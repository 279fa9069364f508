"""Calls of the routing entry points at the edges of what they take (refusals and empty tensors, on the CPU), the
split-size argument, and the routing kernels' assembly."""

import os
import subprocess

import pytest

from test_moe import _lib, _refused
from test_store_hazard import CSRC, _violations

A, B, C, D, E = 0x1000, 0x2000, 0x3000, 0x4000, 0x5000  # never dereferenced: no call below launches


def test_an_output_must_not_be_an_input():
    N, lib = _lib()
    p = N.RouteParams(0, 1, 1.0)
    _refused(-1, lib.mgs_moe_route_bwd(p, 4, 8, 2, A, 1, 8, B, C, A, 8, None), "must not be")
    dis = lambda row=C, rows=D: lib.mgs_moe_dispatch(4, 2, 8, A, 64, 0, B, 64, None, rows, 8, None, row, E, None, 0, None)
    _refused(-1, dis(row=A), "must not be")
    _refused(-1, dis(rows=B), "must not be")
    _refused(-1, lib.mgs_moe_combine(4, 2, 64, 0, A, 8, B, None, B, 64, None), "must not be")
    _refused(-1, lib.mgs_moe_dispatch_bwd(4, 2, 64, 0, A, 8, B, None, B, 64, None, None), "must not be")
    cb = lambda drows: lib.mgs_moe_combine_bwd(4, 2, 64, 0, A, 8, B, 64, C, None, drows, D, None)
    _refused(-1, cb(B), "must not be")
    _refused(-1, cb(C), "must not be")


def test_more_threads_than_a_launch_has():
    N, lib = _lib()
    p = N.RouteParams(0, 1, 1.0)
    many = 1 << 28  # a router workgroup has 16 tokens
    _refused(-2, lib.mgs_moe_route(p, many, 8, 1, A, 0, 8, B, C, None), "too many tokens")
    _refused(-2, lib.mgs_moe_route_bwd(p, many, 8, 1, A, 0, 8, B, C, D, 8, None), "too many tokens")
    wide = 1 << 24  # 2048 BF16 elements and more: a workgroup per token
    _refused(-2, lib.mgs_moe_dispatch(wide, 1, 8, A, 2048, 0, B, 2048, None, C, wide, None, D, E, 0x6000, 1 << 30, None),
             "too many tokens")
    _refused(-2, lib.mgs_moe_combine(wide, 1, 2048, 0, A, 8, B, None, C, 2048, None), "too many tokens")
    _refused(-2, lib.mgs_moe_dispatch_bwd(wide, 1, 2048, 0, A, 8, B, None, C, 2048, None, None), "too many tokens")
    _refused(-2, lib.mgs_moe_combine_bwd(wide, 1, 2048, 0, A, 8, B, 2048, C, None, D, None, None), "too many tokens")


def test_tensors_without_elements_may_be_null():
    N, lib = _lib()
    # no tokens: row_weights has rows, weights [0, topk] has no address (split_sizes is still refused when missing)
    _refused(-1, lib.mgs_moe_dispatch(0, 2, 8, None, 64, 0, None, 64, None, A, 8, B, None, None, None, 0, None), "split_sizes")
    assert lib.mgs_moe_dispatch_bwd(0, 2, 64, 0, None, 8, A, B, None, 64, None, None) == 0
    # no rows: every slot is without one
    assert lib.mgs_moe_combine_bwd(4, 2, 64, 0, A, 0, B, 64, None, None, None, None, None) == 0


def test_split_sizes_beyond_64_bits_are_refused():
    from moe_grouped_scaled_amd import _native as N
    assert N.qtensor_nbytes("mxfp4", False, [5, 3], 64, "data") == 256
    with pytest.raises(OverflowError):
        N.qtensor_nbytes("mxfp4", False, [5, 1 << 64], 64, "data")


def test_routing_kernels_keep_store_data_and_use_no_scratch(tmp_path):
    from moe_grouped_scaled_amd.build import FLAGS, HIPCC
    import re
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    src, flags = os.path.join(CSRC, "moe_route.hip"), [f for f in FLAGS if not f.startswith("-W")]
    run = lambda *a: subprocess.run([HIPCC, *flags, *a, src], check=True, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    run("--cuda-device-only", "-S", "-o", str(tmp_path / "r.s"))
    asm = (tmp_path / "r.s").read_text()
    assert "global_store_dwordx4" in asm
    bad = _violations(asm)
    assert not bad, bad[:5]
    res = run("-c", "-o", str(tmp_path / "r.o"), "-Rpass-analysis=kernel-resource-usage").stdout
    scratch = [int(v) for v in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", res)]
    assert scratch and not any(scratch)
