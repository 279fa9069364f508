"""Weights in 4 bits with a scale (and a zero point) per group, multiplied by BF16 rows: the serving form of the
gated expert block.

`w4_pack` lays weights out once, from a checkpoint's codes, scales and zero points or from what `w4_quantize` makes of
BF16 weights.  The products check their tensors, allocate the outputs that are not given and enqueue the library's
kernels on the tensors' device, on its current stream (or on `stream`, as in `moe`); split sizes and groups as
in `gated`.
"""

import torch

from . import _native as N
from .expert_mlp import GATED
from .gated import _BF16, _F32, _OUT, _check_groups, _gated_act, _given, _groups, _maybe
from .moe import _call, _check, _fail, _int32, _on_stream

_U8 = (torch.uint8,)


class W4Tensor:
    """Packed 4-bit weights [experts, n, k]: `data` (uint8), `shape`, `group`, `zeros` (whether it has zero points)."""

    def __init__(self, data, shape, group, zeros):
        self.shape, self.group, self.zeros = tuple(int(v) for v in shape), int(group), bool(zeros)
        size = _nbytes(*self.shape, self.group, self.zeros)
        if not isinstance(data, torch.Tensor) or data.dtype != torch.uint8 or not data.is_contiguous() or data.numel() != size:
            _fail("data must be a contiguous uint8 tensor of %d bytes", size)
        self.data = data

    @property
    def device(self):
        return self.data.device

    def nbytes(self):
        return self.data.numel()


def _check_w4(what, w, device=None):
    if not isinstance(w, W4Tensor):
        _fail("%s must be a W4Tensor (see w4_pack)", what)
    if device is not None and w.device != device:
        _fail("%s is on %s, expected %s", what, w.device, device)
    return w


def _nbytes(e, n, k, group, zeros):
    _int32("experts", e)
    _int32("group", group)
    size = N.LIB.mgs_w4_nbytes(e, n, k, group, int(zeros))
    if size < 0:
        N._check(int(size))
    return int(size)


def w4_pack(codes, scales, zeros=None, stream=None):
    """A W4Tensor of `codes` uint8 [E, n, k / 2] (two a byte, the even element in the low half), `scales` BF16 [E, n, k /
    group] and `zeros` uint8 of the scales' shape (0 .. 15; 8 everywhere when None): w = (code - zero) * scale."""
    if stream is not None:
        return _on_stream(stream, codes, w4_pack, codes, scales, zeros)
    _check("codes", codes, _U8, 3)
    dev = codes.device
    _check("scales", scales, _BF16, 3, dev)
    e, n, k = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
    ng = scales.shape[2]
    if scales.shape[:2] != codes.shape[:2] or not ng or k % ng:
        _fail("scales has shape %s, which does not fit codes of shape %s", tuple(scales.shape), tuple(codes.shape))
    if zeros is not None:
        _check("zeros", zeros, _U8, 3, dev, shape=scales.shape)
    group = k // ng
    data = torch.empty(_nbytes(e, n, k, group, zeros is not None), dtype=torch.uint8, device=dev)
    _call(dev, N.LIB.mgs_w4_pack, e, n, k, group, codes.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(),
          data.data_ptr())
    return W4Tensor(data, (e, n, k), group, zeros is not None)


def w4_quantize(w, group=128, zeros=True, stream=None):
    """Codes, scales and zero points (None without `zeros`: symmetric) of BF16 weights [E, n, k], in the form `w4_pack`
    takes."""
    if stream is not None:
        return _on_stream(stream, w, w4_quantize, w, group, zeros)
    _int32("group", group)
    _check("w", w, _BF16, 3)
    e, n, k = w.shape
    _nbytes(e, n, k, group, zeros)  # (refuses what does not fit)
    codes = torch.empty((e, n, k // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((e, n, k // group), dtype=torch.bfloat16, device=w.device)
    z = torch.empty(scales.shape, dtype=torch.uint8, device=w.device) if zeros else None
    _call(w.device, N.LIB.mgs_w4_quantize, e, n, k, group, w.data_ptr(), codes.data_ptr(), scales.data_ptr(),
          None if z is None else z.data_ptr())
    return codes, scales, z


def grouped_gemm_w4(split_sizes, x, w, bias=None, y=None, out_dtype=torch.bfloat16, stream=None):
    """y [M, n] = x_g w_g^T + bias for x [M, k] BF16, w a W4Tensor [E, n, k] and bias [E, n] BF16; y is BF16 or FP32
    (allocated as `out_dtype`)."""
    if stream is not None:
        return _on_stream(stream, x, grouped_gemm_w4, split_sizes, x, w, bias, y, out_dtype)
    if out_dtype not in _OUT:
        _fail("out_dtype must be torch.bfloat16 or torch.float32, not %s", out_dtype)
    _check("x", x, _BF16, 2)
    dev = x.device
    e, n, k = _check_w4("w", w, dev).shape
    _check("x", x, _BF16, 2, shape=(x.shape[0], k))
    g = _groups(split_sizes, x.shape[0], e, dev)
    y = _given("y", y, (out_dtype,) if y is None else _OUT, (x.shape[0], n), dev)
    _call(dev, N.LIB.mgs_grouped_gemm_w4, g.ref, n, k, w.group, int(w.zeros), x.data_ptr(), w.data.data_ptr(),
          _maybe("bias", bias, _BF16, (e, n), dev), y.data_ptr(), N.DTYPE[y.dtype])
    return y


def grouped_gated_w4(act, split_sizes, x, w, bias=None, probs=None, h=None, stream=None):
    """h [M, f] = act(gate, up) * probs with [gate | up] = x_g w_g^T + bias in FP32: x [M, k] BF16, w a W4Tensor [E, 2f,
    k], bias [E, 2f] BF16, probs [M] FP32 (1 when None); `act` as in `grouped_gated_fwd`."""
    if stream is not None:
        return _on_stream(stream, x, grouped_gated_w4, act, split_sizes, x, w, bias, probs, h)
    act = _gated_act(act)
    _check("x", x, _BF16, 2)
    dev = x.device
    e, f2, k = _check_w4("w", w, dev).shape
    _check("x", x, _BF16, 2, shape=(x.shape[0], k))
    if f2 % 2:
        _fail("w has %d rows an expert, expected gate and up halves", f2)
    g = _groups(split_sizes, x.shape[0], e, dev)
    h = _given("h", h, _BF16, (x.shape[0], f2 // 2), dev)
    _call(dev, N.LIB.mgs_grouped_gated_w4, act, g.ref, f2 // 2, k, w.group, int(w.zeros), x.data_ptr(), w.data.data_ptr(),
          _maybe("bias", bias, _BF16, (e, f2), dev), _maybe("probs", probs, _F32, (x.shape[0],), dev), h.data_ptr())
    return h


class W4GatedMLP:
    """The gated block of every expert with 4-bit weights, forward only, in place of an `ExpertMLP` in a `MoELayer`
    that serves: w1 a W4Tensor [E, 2F, H] ([gate | up]), w2 [E, H, F], b1 [E, 2F] and b2 [E, H] BF16."""

    grad_x1 = grad_probs = grad_fc1 = grad_fc2 = False

    def __init__(self, kind, w1, w2, b1=None, b2=None, limit=7.0, alpha=1.0, beta=0.0):
        if kind not in GATED:
            _fail("kind must be one of %s, not %r", ", ".join(GATED), kind)
        self.e, self.f_in, self.h = _check_w4("w1", w1).shape
        dev = w1.device
        self.f = self.f_in // 2
        if _check_w4("w2", w2, dev).shape != (self.e, self.h, self.f) or self.f_in % 2:
            _fail("w2 has shape %s, which does not fit w1 of shape %s", w2.shape, w1.shape)
        _maybe("b1", b1, _BF16, (self.e, self.f_in), dev)
        _maybe("b2", b2, _BF16, (self.e, self.h), dev)
        self.kind, self.fmt = kind, "w4"
        self.w1, self.w2, self.b1, self.b2 = w1, w2, b1, b2
        self.act = N.act_params(kind, limit=limit, alpha=alpha, beta=beta)
        self.ctx = None

    def forward(self, x1, probs, splits):
        """x1 [M, H] BF16, probs [M] FP32 or None, `splits` host split sizes or an N.DeviceGroups -> [M, H] BF16."""
        if isinstance(splits, N.DeviceGroups):
            # (all of it ahead of the update, whose kernel would write a table on another device from this one)
            _check("x1", x1, _BF16, 2, self.w1.device)
            _check_groups(splits, x1.shape[0], self.e, x1.device)
            with torch.cuda.device(x1.device):
                splits.update()
        h = grouped_gated_w4(self.act, splits, x1, self.w1, self.b1, probs)
        self.ctx = {}  # nothing is kept; MoELayer marks it
        return grouped_gemm_w4(splits, h, self.w2, self.b2)

    def backward(self, dy2):
        _fail("4-bit weights have no backward")
