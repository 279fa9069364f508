"""The gated expert block in BF16: gate and up projection, activation, product and second linear, and back.

The functions check their tensors, allocate the outputs that are not given and enqueue the library's kernels on
the tensors' device, on its current stream (or on `stream`, as in `moe`).  `split_sizes` are host row counts or an
`_native.DeviceGroups`, whose capacity is then the tensors' row count; rows past the last used one are neither
read nor written.  Tensors are contiguous; an output must not be or overlap another tensor of its call.

`GatedMLP` is the block with its backward, in place of an `ExpertMLP` in a `MoELayer` where nothing is quantized.
"""

import torch

from . import _native as N
from .expert_mlp import GATED
from .moe import _call, _check, _fail, _on_stream

_BF16, _F32 = (torch.bfloat16,), (torch.float32,)
_OUT = (torch.bfloat16, torch.float32)


def _check_groups(split_sizes, rows, experts, device):
    """The groups must cover `rows` rows of `experts` experts on `device`."""
    n = len(split_sizes)
    if n != experts:
        _fail("split_sizes has %d entries, the weights %d experts", n, experts)
    if isinstance(split_sizes, N.DeviceGroups):
        if split_sizes.max_rows != rows:
            _fail("with device-resident split sizes the tensors have the capacity's %d rows (got %d)",
                  split_sizes.max_rows, rows)
        if split_sizes.table.device != device:
            _fail("the split sizes are on %s, the tensors on %s", split_sizes.table.device, device)
    elif sum(split_sizes) != rows:
        _fail("the split sizes add up to %d, the tensors have %d rows", sum(split_sizes), rows)


def _groups(split_sizes, rows, experts, device):
    """The library's view of the groups (see _check_groups)."""
    _check_groups(split_sizes, rows, experts, device)
    return N._GroupsArg(split_sizes)


def _gated_act(act):
    """mgs_act_params of a gated kind from its name or from `act_params`."""
    if isinstance(act, str):
        if act not in GATED:
            _fail("act must be one of %s, not %r", ", ".join(GATED), act)
        return N.act_params(act)
    if not isinstance(act, N.ActParams):
        _fail("act must be a name or act_params(...)")
    return act


def _given(what, t, dtypes, shape, device):
    """The output `what`, allocated if it is None."""
    if t is None:
        return torch.empty(shape, dtype=dtypes[0], device=device)
    return _check(what, t, dtypes, len(shape), device, shape=shape)


def _maybe(what, t, dtypes, shape, device):
    return None if t is None else _check(what, t, dtypes, len(shape), device, shape=shape).data_ptr()


def grouped_gemm_bf16(mode, split_sizes, a, b, c=None, bias=None, accumulate=False, out_dtype=torch.bfloat16, stream=None):
    """Grouped product of BF16 tensors in FP32: "fprop" c = a b_g^T (b [E, n, k]), "dgrad" c = a b_g (b [E, k, n]), both
    with an optional bias [E, n], or "wgrad" c_g = a_g^T b_g (a [M, m], b [M, n], c [E, m, n]).  c is BF16 or FP32
    (allocated as `out_dtype`); `accumulate` adds into an FP32 c."""
    if stream is not None:
        return _on_stream(stream, a, grouped_gemm_bf16, mode, split_sizes, a, b, c, bias, accumulate, out_dtype)
    if mode not in N.GEMM_MODE:
        _fail("mode must be one of %s, not %r", ", ".join(N.GEMM_MODE), mode)
    if out_dtype not in _OUT:
        _fail("out_dtype must be torch.bfloat16 or torch.float32, not %s", out_dtype)
    if accumulate and c is None:
        _fail("accumulate needs a c to add into")
    _check("a", a, _BF16, 2)
    dev, rows = a.device, a.shape[0]
    if mode == "wgrad":
        _check("b", b, _BF16, 2, dev)
        if b.shape[0] != rows:
            _fail("b has %d rows, expected %d", b.shape[0], rows)
        e, m, n, k = len(split_sizes), a.shape[1], b.shape[1], rows
        shape = (e, m, n)
        if bias is not None:
            _fail("bias is not defined for wgrad")
    else:
        _check("b", b, _BF16, 3, dev)
        e, m, k = b.shape[0], rows, a.shape[1]
        n = b.shape[1] if mode == "fprop" else b.shape[2]
        if b.shape[2 if mode == "fprop" else 1] != k:
            _fail("b has shape %s, which does not fit rows of width %d", tuple(b.shape), k)
        shape = (rows, n)
    g = _groups(split_sizes, rows, e, dev)
    c = _given("c", c, (out_dtype,) if c is None else _OUT, shape, dev)
    _call(dev, N.LIB.mgs_grouped_gemm_bf16, N.GEMM_MODE[mode], g.ref, m, n, k, a.data_ptr(), b.data_ptr(), c.data_ptr(),
          N.DTYPE[c.dtype], _maybe("bias", bias, _BF16, (e, n), dev), int(bool(accumulate)))
    return c


def grouped_gated_fwd(act, split_sizes, x, w, bias=None, probs=None, h=None, pre=None, stream=None):
    """h = act(gate, up) * probs with [gate | up] = x w_g^T + bias in FP32: x [M, k], w [E, 2f, k], bias [E, 2f], probs
    [M] FP32 (1 when None).  `act`: "swiglu", "clamped_swiglu", "glu" or `act_params(...)` of one.  `pre` [M, 2f],
    FP32 or BF16, receives [gate | up] for the backward.  Returns h [M, f]."""
    if stream is not None:
        return _on_stream(stream, x, grouped_gated_fwd, act, split_sizes, x, w, bias, probs, h, pre)
    act = _gated_act(act)
    _check("x", x, _BF16, 2)
    dev, (rows, k) = x.device, x.shape
    _check("w", w, _BF16, 3, dev)
    e, f2 = w.shape[0], w.shape[1]
    if w.shape[2] != k:
        _fail("w has rows of width %d, x of width %d", w.shape[2], k)
    if f2 % 2:
        _fail("w has %d rows an expert, expected gate and up halves", f2)
    g = _groups(split_sizes, rows, e, dev)
    h = _given("h", h, _BF16, (rows, f2 // 2), dev)
    _call(dev, N.LIB.mgs_grouped_gated_fwd, act, g.ref, f2 // 2, k, x.data_ptr(), w.data_ptr(),
          _maybe("bias", bias, _BF16, (e, f2), dev), _maybe("probs", probs, _F32, (rows,), dev), h.data_ptr(),
          _maybe("pre", pre, _OUT, (rows, f2), dev), N.DTYPE[torch.float32 if pre is None else pre.dtype])
    return h


def grouped_gated_bwd_workspace_bytes(split_sizes, f):
    g = N._GroupsArg(split_sizes)
    n = N.LIB.mgs_grouped_gated_bwd_workspace_bytes(g.ref, int(f))
    if n < 0:
        N._check(int(n))
    return int(n)


def grouped_gated_bwd(act, split_sizes, dy, w2, pre, probs=None, dpre=None, h=None, dprobs=None, workspace=None, stream=None):
    """Backward of the second linear and the activation: with da = dy w2_g (w2 [E, n, f]) in FP32, dpre [M, 2f] = da *
    probs * the activation's derivatives at `pre`; `h` [M, f] receives the second linear's input again, `dprobs`
    [M] FP32 the sum of da * act(pre).  Returns dpre."""
    if stream is not None:
        return _on_stream(stream, dy, grouped_gated_bwd, act, split_sizes, dy, w2, pre, probs, dpre, h, dprobs, workspace)
    act = _gated_act(act)
    _check("dy", dy, _BF16, 2)
    dev, (rows, n) = dy.device, dy.shape
    _check("w2", w2, _BF16, 3, dev)
    e, f = w2.shape[0], w2.shape[2]
    if w2.shape[1] != n:
        _fail("w2 has %d rows an expert, dy is %d wide", w2.shape[1], n)
    _check("pre", pre, _OUT, 2, dev, shape=(rows, 2 * f))
    g = _groups(split_sizes, rows, e, dev)
    dpre = _given("dpre", dpre, _BF16, (rows, 2 * f), dev)
    dp = _maybe("dprobs", dprobs, _F32, (rows,), dev)
    ws, wb = None, 0
    if dp is not None and rows:
        if workspace is None:
            workspace = torch.empty(grouped_gated_bwd_workspace_bytes(split_sizes, f), dtype=torch.uint8, device=dev)
        ws, wb = _check("workspace", workspace, (torch.uint8,), 1, dev).data_ptr(), workspace.numel()
    _call(dev, N.LIB.mgs_grouped_gated_bwd, act, g.ref, f, n, dy.data_ptr(), w2.data_ptr(), pre.data_ptr(), N.DTYPE[pre.dtype],
          _maybe("probs", probs, _F32, (rows,), dev), dpre.data_ptr(), _maybe("h", h, _BF16, (rows, f), dev), dp, ws, wb)
    return dpre


def _marks(*tensors):
    """Of each tensor that is kept by reference, torch's count of its in-place changes.  None, which nothing is compared
    with: for a part of a larger storage (whose other parts may change), for a tensor without a count, and inside a
    captured graph, whose buffers change between replays."""
    if torch.cuda.is_current_stream_capturing():
        return (None,) * len(tensors)
    return tuple(None if t is None or t.is_inference() or t.untyped_storage().nbytes() != t.numel() * t.element_size()
                 else t._version for t in tensors)


def _unchanged(what, t, mark, since):
    if mark is not None and t._version != mark:
        _fail("%s was changed in place since the %s: it is kept, not copied, for the gradients", what, since)


class GatedMLP:
    """The gated block of every expert in BF16, forward and backward, with the interface of `ExpertMLP`.

    kind "swiglu", "clamped_swiglu" or "glu"; w1 [E, 2F, H] ([gate | up]), b1 [E, 2F], w2 [E, H, F], b2 [E, H], all BF16.
    forward(x1 [M, H], probs [M] FP32 or None, split_sizes) -> y2 [M, H]; backward(dy2) -> dx1 and dprobs and, unless
    `delay_wgrad`, dw1, dw2 (of `dw_dtype`, FP32 by default) and db1, db2 (FP32); each gradient is
    requested by grad_x1, grad_probs, grad_fc1, grad_fc2, and what only an unrequested one needs is neither
    computed nor kept.  The forward keeps [gate | up] in `save_dtype`: FP32, or BF16 for half the memory (the
    gradients are then those at the rounded values, and carry that rounding's error beside their own), and with `recompute`
    regenerates the second linear's input from it in the backward instead of keeping that too (from BF16, the regenerated
    rows differ from the forward's by the rounding of [gate | up]).  Rows are one captured step's own:
    every forward allocates its outputs.

    With `delay_wgrad` the weight and bias gradients of a backward are computed by backward_dw(), before the next
    backward (which is refused while they are pending).  x1, probs and dy2 are kept, not copied (an `ExpertMLP` keeps
    quantized copies): they, and the split sizes of a DeviceGroups, stay as they are until the gradients that need them are
    computed, x1 and dy2 until backward_dw().  An in-place change by torch of a tensor that fills its storage is refused;
    a change of a part of a larger buffer, by a kernel that is given the address, or by a graph's replay is not seen."""

    def __init__(self, kind, w1, w2, b1=None, b2=None, recompute=False, delay_wgrad=False, limit=7.0, alpha=1.0, beta=0.0,
                 grad_x1=True, grad_probs=True, grad_fc1=True, grad_fc2=True, dw_dtype=torch.float32,
                 save_dtype=torch.float32):
        if kind not in GATED:
            _fail("kind must be one of %s, not %r", ", ".join(GATED), kind)
        if dw_dtype not in _OUT:
            _fail("dw_dtype must be torch.bfloat16 or torch.float32, not %s", dw_dtype)
        if save_dtype not in _OUT:
            _fail("save_dtype must be torch.bfloat16 or torch.float32, not %s", save_dtype)
        _check("w1", w1, _BF16, 3)
        self.e, self.f_in, self.h = w1.shape
        if self.f_in % 2:
            _fail("w1 has %d rows an expert, expected gate and up halves", self.f_in)
        self.f = self.f_in // 2
        dev = w1.device
        _check("w2", w2, _BF16, 3, dev, shape=(self.e, self.h, self.f))
        _maybe("b1", b1, _BF16, (self.e, self.f_in), dev)
        _maybe("b2", b2, _BF16, (self.e, self.h), dev)
        self.kind, self.fmt, self.dw_dtype, self.save_dtype = kind, "bf16", dw_dtype, save_dtype
        self.w1, self.w2, self.b1, self.b2 = w1, w2, b1, b2
        self.recompute, self.delay_wgrad = bool(recompute), bool(delay_wgrad)
        self.grad_x1, self.grad_probs, self.grad_fc1, self.grad_fc2 = grad_x1, grad_probs, grad_fc1, grad_fc2
        self.grad_below_fc2 = grad_x1 or grad_probs or grad_fc1
        self.act = N.act_params(kind, limit=limit, alpha=alpha, beta=beta)
        self.ctx = None
        self.pending_wgrad = None

    def forward(self, x1, probs, splits):
        """`splits`: host split sizes, or an N.DeviceGroups, whose offsets the step computes first, so that a captured
        graph of it follows the split sizes held in the device tensor."""
        _check("x1", x1, _BF16, 2, self.w1.device)
        if x1.shape[1] != self.h:
            _fail("x1 has rows of width %d, w1 of width %d", x1.shape[1], self.h)
        if isinstance(splits, N.DeviceGroups):
            # (ahead of the update, whose kernel would write a table on another device from this one)
            _check_groups(splits, x1.shape[0], self.e, x1.device)
        with torch.cuda.device(x1.device):
            if isinstance(splits, N.DeviceGroups):
                splits.update()
            else:
                splits = [int(s) for s in splits]
            keep_pre = self.grad_below_fc2 or (self.grad_fc2 and self.recompute)
            pre = torch.empty((x1.shape[0], self.f_in), dtype=self.save_dtype, device=x1.device) if keep_pre else None
            a = grouped_gated_fwd(self.act, splits, x1, self.w1, self.b1, probs, pre=pre)
            y2 = grouped_gemm_bf16("fprop", splits, a, self.w2, bias=self.b2)
            x1 = x1 if self.grad_fc1 else None
            marks = _marks(x1, probs) if keep_pre else (None, None)
        self.ctx = dict(splits=splits, probs=probs, pre=pre, x1=x1, a=a if self.grad_fc2 and not self.recompute else None,
                        marks=marks)
        return y2

    def backward(self, dy2):
        c = self.ctx
        if c is None:
            _fail("backward() without a forward")
        if self.pending_wgrad is not None and (self.grad_fc1 or self.grad_fc2):
            _fail("the weight gradients of the last backward() are still to be computed: backward_dw() (or drop them: "
                  "pending_wgrad = None)")
        splits, pre, a = c["splits"], c["pre"], c["a"]
        x1_mark, probs_mark = c["marks"]
        _unchanged("x1", c["x1"], x1_mark, "forward")
        _unchanged("probs", c["probs"], probs_mark, "forward")
        m = sum(splits) if isinstance(splits, list) else splits.max_rows
        _check("dy2", dy2, _BF16, 2, self.w1.device, shape=(m, self.h))
        grads = {}
        dpre = None
        with torch.cuda.device(dy2.device):
            regenerate = self.grad_fc2 and self.recompute
            if regenerate:
                a = torch.empty((m, self.f), dtype=torch.bfloat16, device=dy2.device)
            if self.grad_below_fc2 or regenerate:
                dprobs = None
                if self.grad_probs:
                    dprobs = grads["dprobs"] = torch.empty(m, dtype=torch.float32, device=dy2.device)
                dpre = grouped_gated_bwd(self.act, splits, dy2, self.w2, pre, c["probs"], h=a if regenerate else None,
                                         dprobs=dprobs)
            if self.grad_x1:
                grads["dx1"] = grouped_gemm_bf16("dgrad", splits, dpre, self.w1)
            dy2 = dy2 if self.grad_fc2 else None
            dy2_mark = _marks(dy2)[0] if self.delay_wgrad else None
        self.pending_wgrad = dict(splits=splits, dy2=dy2, a=a, dpre=dpre if self.grad_fc1 else None, x1=c["x1"], x1_mark=x1_mark,
                                  dy2_mark=dy2_mark)
        self.ctx = None
        if not self.delay_wgrad:
            try:
                grads.update(self.backward_dw())
            finally:
                self.pending_wgrad = None
        return grads

    def backward_dw(self, dw1=None, dw2=None, accumulate=False):
        """Weight gradients (into dw1, dw2 if given, adding with `accumulate`) and bias gradients of the last backward."""
        p = self.pending_wgrad
        if p is None:
            _fail("backward_dw() without a pending backward")
        splits, out = p["splits"], {}
        _unchanged("x1", p["x1"], p["x1_mark"], "forward")
        _unchanged("dy2", p["dy2"], p["dy2_mark"], "backward")
        # (all is checked and allocated before the first launch: a call that fails has added nothing)
        if self.grad_fc2:
            out["dw2"] = self._weight_grad("dw2", dw2, (self.e, self.h, self.f), accumulate)
        if self.grad_fc1:
            out["dw1"] = self._weight_grad("dw1", dw1, (self.e, self.f_in, self.h), accumulate)
        for name, bias in (("db2", self.b2 if self.grad_fc2 else None), ("db1", self.b1 if self.grad_fc1 else None)):
            if bias is not None:
                out[name] = torch.empty(bias.shape, dtype=torch.float32, device=bias.device)
        with torch.cuda.device(self.w1.device):
            if self.grad_fc2:
                grouped_gemm_bf16("wgrad", splits, p["dy2"], p["a"], out["dw2"], accumulate=accumulate)
            if "db2" in out:
                N.grouped_col_sum(splits, self.h, p["dy2"], out["db2"])
            if self.grad_fc1:
                grouped_gemm_bf16("wgrad", splits, p["dpre"], p["x1"], out["dw1"], accumulate=accumulate)
            if "db1" in out:
                N.grouped_col_sum(splits, self.f_in, p["dpre"], out["db1"])
        self.pending_wgrad = None
        return out

    def _weight_grad(self, name, t, shape, accumulate):
        """The weight gradient `name` to write or, with `accumulate`, to add into: `t`, or a new one."""
        if accumulate and t is None:
            _fail("accumulate needs a %s to add into", name)
        t = _given(name, t, (self.dw_dtype,) if t is None else _F32 if accumulate else _OUT, shape, self.w1.device)
        if t.data_ptr() % 16:
            _fail("%s must be 16-byte aligned", name)
        return t
