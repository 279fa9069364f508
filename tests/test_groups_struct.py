"""The binding's `Groups` is made by callers of the C entry points too: split sizes as a typed pointer, an array or
nothing, and the same sizes from every form of them."""

import ctypes

import numpy as np


def test_split_sizes_of_every_form():
    from moe_grouped_scaled_amd import _native as N
    sizes = [64, 0, 37]
    arr = (ctypes.c_int64 * 3)(*sizes)
    held = np.array(sizes, dtype=np.int64)
    p64 = ctypes.POINTER(ctypes.c_int64)
    want = N.qtensor_nbytes("mxfp8", True, sizes, 64, "data")
    assert want == (128 + 128) * 64
    for s in (arr, ctypes.cast(arr, p64), held.ctypes.data_as(p64)):
        g = N.Groups(3, s, 0, None)
        assert g.split_sizes[2] == 37
        assert N.LIB.mgs_qtensor_nbytes(0, 1, ctypes.byref(g), 64, 0) == want
        assert N.LIB.mgs_qtensor_nbytes(0, 1, g, 64, 0) == want
    for form in (tuple(sizes), held, held.astype(np.int32), np.int64(sizes).tolist(), [np.int64(v) for v in sizes], np.repeat(held, 2)[::2]):
        assert N.qtensor_nbytes("mxfp8", True, form, 64, "data") == want
        assert N._GroupsArg(form).struct.split_sizes[2] == 37
    assert not N.Groups(3, None, 128, 0x1000).split_sizes
