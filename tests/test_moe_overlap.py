"""No output of a routing call may be, or overlap, another tensor of it: workgroups read and write in any order.  Every
pair of every call is refused on the host, before a launch (nothing here is dereferenced)."""

import itertools

import pytest

from test_moe import _lib, _refused

T, K, E, H, ROWS = 4, 2, 8, 64, 8   # bytes: below
I, O = "in", "out"
# tensors of each call: name -> (in or out, bytes)
CALLS = {
    "route": dict(logits=(I, T * E * 4), idx=(O, T * K * 4), weights=(O, T * K * 4)),
    "route_bwd": dict(logits=(I, T * E * 4), idx=(I, T * K * 4), dweights=(I, T * K * 4), dlogits=(O, T * E * 4)),
    "dispatch": dict(idx=(I, T * K * 4), x=(I, T * H * 4), weights=(I, T * K * 4), rows=(O, T * K * H * 4), row_weights=(O, ROWS * 4),
                     row=(O, T * K * 4), splits=(O, E * 8)),
    "dispatch_bwd": dict(row=(I, T * K * 4), drows=(I, ROWS * H * 4), drow_weights=(I, ROWS * 4), dx=(O, T * H * 4), dweights=(O, T * K * 4)),
    "combine": dict(row=(I, T * K * 4), rows=(I, ROWS * H * 4), weights=(I, T * K * 4), y=(O, T * H * 4)),
    "combine_bwd": dict(row=(I, T * K * 4), dy=(I, T * H * 4), rows=(I, ROWS * H * 4), weights=(I, T * K * 4), drows=(O, ROWS * H * 4),
                        dweights=(O, T * K * 4)),
}
PAIRS = [(call, a, b) for call, t in CALLS.items() for a, b in itertools.permutations(t, 2)
         if t[a][0] == O and (t[b][0] == I or list(t).index(a) < list(t).index(b))]


def _call(name, p):
    N, lib = _lib()
    rp = N.RouteParams(0, 1, 1.0)
    if name == "route":
        return lib.mgs_moe_route(rp, T, E, K, p["logits"], 1, E, p["idx"], p["weights"], None)
    if name == "route_bwd":
        return lib.mgs_moe_route_bwd(rp, T, E, K, p["logits"], 1, E, p["idx"], p["dweights"], p["dlogits"], E, None)
    if name == "dispatch":
        return lib.mgs_moe_dispatch(T, K, E, p["idx"], H, 1, p["x"], H, p["weights"], p["rows"], ROWS, p["row_weights"], p["row"],
                                    p["splits"], None, 0, None)
    if name == "dispatch_bwd":
        return lib.mgs_moe_dispatch_bwd(T, K, H, 1, p["row"], ROWS, p["drows"], p["drow_weights"], p["dx"], H, p["dweights"], None)
    if name == "combine":
        return lib.mgs_moe_combine(T, K, H, 1, p["row"], ROWS, p["rows"], p["weights"], p["y"], H, None)
    return lib.mgs_moe_combine_bwd(T, K, H, 1, p["row"], ROWS, p["dy"], H, p["rows"], p["weights"], p["drows"], p["dweights"], None)


@pytest.mark.parametrize("call,a,b", PAIRS)
def test_same_or_overlapping(call, a, b):
    tensors = CALLS[call]
    at = {n: 0x10000 * (i + 1) for i, n in enumerate(tensors)}
    _refused(-1, _call(call, dict(at, **{a: at[b]})), "must not be")
    _refused(-1, _call(call, dict(at, **{a: at[b] + tensors[b][1] - 4})), "must not be")   # starts in its last element
    _refused(-1, _call(call, dict(at, **{a: at[b] - tensors[a][1] + 4})), "must not be")   # ends in its first


def test_strided_rows_and_the_workspace():
    N, lib = _lib()
    rp = N.RouteParams(0, 1, 1.0)
    A, B, C, D, F = (0x1000000 * i for i in range(1, 6))
    # rows E wide, 2 E apart: the same start is refused
    _refused(-1, lib.mgs_moe_route_bwd(rp, T, E, K, A, 1, 2 * E, B, C, A, 2 * E, None), "must not be")
    # and one that starts in the other's first row
    _refused(-1, lib.mgs_moe_route_bwd(rp, T, E, K, A, 1, 2 * E, B, C, A + 4 * (E - 1), 2 * E, None), "must not be")
    need = lib.mgs_moe_dispatch_workspace_bytes(4000, 2, E)
    for ws in (A, B, C, A + 4 * 8000 - 4):
        _refused(-1, lib.mgs_moe_dispatch(4000, 2, E, A, H, 1, None, 0, None, None, 0, None, B, C, ws, need, None), "must not be")
