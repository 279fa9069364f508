"""Routing around the expert MLP: router, dispatch into expert order, combine, their gradients, and the layer.

The functions check their tensors, allocate the outputs that are not given and enqueue the library's
kernels on the tensors' device (its current stream, or `stream`).  Nothing synchronises: the split sizes
stay in device memory, where `_native.DeviceGroups` takes them, so a captured graph follows the routing.

A slot is one (token, choice) pair, numbered token * topk + choice; a slot without an expert has expert -1
and row -1.
"""

import torch

from . import _native as N


def _fail(msg, *args):
    raise ValueError(msg % args if args else msg)


def _check(what, t, dtypes, ndim, device=None, contiguous=True):
    """A CUDA tensor of one of `dtypes`, `ndim` dimensions and unit column stride (rows contiguous when
    `contiguous`), on `device`."""
    if not isinstance(t, torch.Tensor):
        _fail("%s must be a tensor", what)
    if t.dtype not in dtypes:
        _fail("%s has type %s, expected %s", what, t.dtype, " or ".join(str(d) for d in dtypes))
    if t.dim() != ndim:
        _fail("%s has %d dimensions, expected %d", what, t.dim(), ndim)
    if contiguous:
        if not t.is_contiguous():
            _fail("%s must be contiguous", what)
    elif t.numel() and (t.stride(1) != 1 and t.shape[1] > 1 or t.stride(0) < t.shape[1] and t.shape[0] > 1):
        _fail("%s must have unit column stride and rows that do not overlap (strides %s)", what, t.stride())
    if not t.is_cuda:
        _fail("%s must be on a GPU", what)
    if device is not None and t.device != device:
        _fail("%s is on %s, expected %s", what, t.device, device)
    return t


def _shape(what, t, shape):
    if tuple(t.shape) != tuple(shape):
        _fail("%s has shape %s, expected %s", what, tuple(t.shape), tuple(shape))


def _ld(t):
    """Row stride in elements (a single row may carry any stride)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


class _On:
    """The tensors' device as the current one for the launch, and its stream handle."""

    def __init__(self, device, stream):
        self.device, self.stream, self.guard = device, stream, None

    def __enter__(self):
        if self.device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()
        return N._stream(self.stream)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


_FLOATS = (torch.bfloat16, torch.float32)
_I32, _I64, _F32 = (torch.int32,), (torch.int64,), (torch.float32,)


def _params(score, renormalize, scale):
    if score not in N.SCORE:
        _fail("score must be one of %s, not %r", ", ".join(N.SCORE), score)
    return N.RouteParams(N.SCORE[score], int(bool(renormalize)), float(scale))


def moe_route(logits, topk, score="softmax", renormalize=True, scale=1.0, expert_idx=None, weights=None, stream=None):
    """The topk largest of each token's `logits` [tokens, experts] (BF16 or FP32) in descending order, equal
    ones by expert, and their weights: `scale` times the softmax over all experts or the sigmoid, divided
    by the picked ones' sum with `renormalize`.  Experts at -inf are never picked.  Returns
    (expert_idx int32, weights FP32), both [tokens, topk]."""
    _check("logits", logits, _FLOATS, 2, contiguous=False)
    t, e = logits.shape
    dev = logits.device
    if expert_idx is None:
        expert_idx = torch.empty((t, topk), dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty((t, topk), dtype=torch.float32, device=dev)
    _shape("expert_idx", _check("expert_idx", expert_idx, _I32, 2, dev), (t, topk))
    _shape("weights", _check("weights", weights, _F32, 2, dev), (t, topk))
    p = _params(score, renormalize, scale)
    with _On(dev, stream) as s:
        N._check(N.LIB.mgs_moe_route(p, t, e, topk, logits.data_ptr(), N.DTYPE[logits.dtype], _ld(logits),
                                     expert_idx.data_ptr(), weights.data_ptr(), s))
    return expert_idx, weights


def moe_route_bwd(logits, expert_idx, dweights, score="softmax", renormalize=True, scale=1.0, dlogits=None, stream=None):
    """The logits' gradient of `moe_route`'s weights (every element of dlogits is written)."""
    _check("logits", logits, _FLOATS, 2, contiguous=False)
    t, e = logits.shape
    dev = logits.device
    _check("expert_idx", expert_idx, _I32, 2, dev)
    k = expert_idx.shape[1]
    _shape("expert_idx", expert_idx, (t, k))
    _shape("dweights", _check("dweights", dweights, _F32, 2, dev), (t, k))
    if dlogits is None:
        dlogits = torch.empty((t, e), dtype=logits.dtype, device=dev)
    _shape("dlogits", _check("dlogits", dlogits, (logits.dtype,), 2, dev, contiguous=False), (t, e))
    p = _params(score, renormalize, scale)
    with _On(dev, stream) as s:
        N._check(N.LIB.mgs_moe_route_bwd(p, t, e, k, logits.data_ptr(), N.DTYPE[logits.dtype], _ld(logits),
                                         expert_idx.data_ptr(), dweights.data_ptr(), dlogits.data_ptr(), _ld(dlogits), s))
    return dlogits


def moe_dispatch_workspace_bytes(tokens, topk, num_experts):
    n = N.LIB.mgs_moe_dispatch_workspace_bytes(tokens, topk, num_experts)
    if n < 0:
        N._check(int(n))
    return int(n)


def moe_dispatch(expert_idx, num_experts, x=None, rows=None, weights=None, row_weights=None, row_of_slot=None,
                 split_sizes=None, workspace=None, stream=None):
    """Sorts the slots by expert (stable) and copies the token rows there: rows[row_of_slot[t, c]] = x[t], and
    with `weights` [tokens, topk] row_weights[row_of_slot[t, c]] = weights[t, c].  `rows` has at least
    tokens * topk rows; those past the last used one stay as they are.  Without `x` only the sort.  Returns
    (row_of_slot int32 [tokens, topk], split_sizes int64 [num_experts]).  A workspace given here must not be
    shared with a call that may run at the same time."""
    _check("expert_idx", expert_idx, _I32, 2)
    t, k = expert_idx.shape
    dev = expert_idx.device
    need = moe_dispatch_workspace_bytes(t, k, num_experts)
    if row_of_slot is None:
        row_of_slot = torch.empty((t, k), dtype=torch.int32, device=dev)
    if split_sizes is None:
        split_sizes = torch.empty(num_experts, dtype=torch.int64, device=dev)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _shape("row_of_slot", _check("row_of_slot", row_of_slot, _I32, 2, dev), (t, k))
    _shape("split_sizes", _check("split_sizes", split_sizes, _I64, 1, dev), (num_experts,))
    _check("workspace", workspace, (torch.uint8,), 1, dev)
    h, dt, ldx, xp, rp, n, wp, rwp = 0, 0, 0, None, None, 0, None, None
    if x is not None or rows is not None or weights is not None or row_weights is not None:
        if x is None or rows is None:
            _fail("x and rows go together (and weights need them)")
        _check("x", x, _FLOATS, 2, dev, contiguous=False)
        _check("rows", rows, (x.dtype,), 2, dev)
        h, dt, ldx, n = x.shape[1], N.DTYPE[x.dtype], _ld(x), rows.shape[0]
        _shape("x", x, (t, h))
        _shape("rows", rows, (n, h))
        xp, rp = x.data_ptr(), rows.data_ptr()
        if (weights is None) != (row_weights is None):
            _fail("weights and row_weights go together")
        if weights is not None:
            _shape("weights", _check("weights", weights, _F32, 2, dev), (t, k))
            _shape("row_weights", _check("row_weights", row_weights, _F32, 1, dev), (n,))
            wp, rwp = weights.data_ptr(), row_weights.data_ptr()
    with _On(dev, stream) as s:
        N._check(N.LIB.mgs_moe_dispatch(t, k, num_experts, expert_idx.data_ptr(), h, dt, xp, ldx, wp, rp, n, rwp,
                                        row_of_slot.data_ptr(), split_sizes.data_ptr(), workspace.data_ptr(),
                                        workspace.numel(), s))
    return row_of_slot, split_sizes


def _slots_and_rows(row_of_slot, rows, name="rows"):
    _check("row_of_slot", row_of_slot, _I32, 2)
    _check(name, rows, _FLOATS, 2, row_of_slot.device)
    return row_of_slot.shape[0], row_of_slot.shape[1], rows.shape[1], rows.shape[0], row_of_slot.device


def moe_dispatch_bwd(row_of_slot, drows, drow_weights=None, dx=None, dweights=None, stream=None):
    """Gradient of the dispatch: dx[t] = the sum of the token's drows, and with `drow_weights` (FP32, one a row)
    dweights[t, c] = drow_weights[row_of_slot[t, c]].  Returns (dx, dweights or None)."""
    t, k, h, n, dev = _slots_and_rows(row_of_slot, drows, "drows")
    if dx is None:
        dx = torch.empty((t, h), dtype=drows.dtype, device=dev)
    _shape("dx", _check("dx", dx, (drows.dtype,), 2, dev, contiguous=False), (t, h))
    dwp = gwp = None
    if drow_weights is not None:
        _shape("drow_weights", _check("drow_weights", drow_weights, _F32, 1, dev), (n,))
        if dweights is None:
            dweights = torch.empty((t, k), dtype=torch.float32, device=dev)
        _shape("dweights", _check("dweights", dweights, _F32, 2, dev), (t, k))
        gwp, dwp = drow_weights.data_ptr(), dweights.data_ptr()
    elif dweights is not None:
        _fail("dweights needs drow_weights")
    with _On(dev, stream) as s:
        N._check(N.LIB.mgs_moe_dispatch_bwd(t, k, h, N.DTYPE[drows.dtype], row_of_slot.data_ptr(), n, drows.data_ptr(),
                                            gwp, dx.data_ptr(), _ld(dx), dwp, s))
    return dx, dweights


def moe_combine(row_of_slot, rows, weights=None, y=None, stream=None):
    """y[t] = the sum over the token's slots of weights[t, c] * rows[row_of_slot[t, c]] (weights 1 when None),
    in FP32 with one rounding."""
    t, k, h, n, dev = _slots_and_rows(row_of_slot, rows)
    if y is None:
        y = torch.empty((t, h), dtype=rows.dtype, device=dev)
    _shape("y", _check("y", y, (rows.dtype,), 2, dev, contiguous=False), (t, h))
    if weights is not None:
        _shape("weights", _check("weights", weights, _F32, 2, dev), (t, k))
    with _On(dev, stream) as s:
        N._check(N.LIB.mgs_moe_combine(t, k, h, N.DTYPE[rows.dtype], row_of_slot.data_ptr(), n, rows.data_ptr(),
                                       None if weights is None else weights.data_ptr(), y.data_ptr(), _ld(y), s))
    return y


def moe_combine_bwd(row_of_slot, dy, drows=None, rows=None, weights=None, dweights=None, stream=None):
    """Gradient of the combine: drows[row_of_slot[t, c]] = weights[t, c] * dy[t] (rows no slot has stay as they
    are), and with `rows`, the forward's input, dweights[t, c] = <dy[t], rows[row_of_slot[t, c]]>, which is
    returned (else None)."""
    _check("row_of_slot", row_of_slot, _I32, 2)
    dev = row_of_slot.device
    t, k = row_of_slot.shape
    _check("dy", dy, _FLOATS, 2, dev, contiguous=False)
    h = dy.shape[1]
    _shape("dy", dy, (t, h))
    n = None
    for name, v in (("drows", drows), ("rows", rows)):
        if v is not None:
            _check(name, v, (dy.dtype,), 2, dev)
            n = v.shape[0] if n is None else n
            _shape(name, v, (n, h))
    if n is None:
        _fail("drows or rows is needed")
    if rows is not None and dweights is None:
        dweights = torch.empty((t, k), dtype=torch.float32, device=dev)
    for name, v in (("weights", weights), ("dweights", dweights)):
        if v is not None:
            _shape(name, _check(name, v, _F32, 2, dev), (t, k))
    ptr = lambda v: None if v is None else v.data_ptr()
    with _On(dev, stream) as s:
        N._check(N.LIB.mgs_moe_combine_bwd(t, k, h, N.DTYPE[dy.dtype], row_of_slot.data_ptr(), n, dy.data_ptr(), _ld(dy),
                                           ptr(rows), ptr(weights), ptr(drows), ptr(dweights), s))
    return dweights


class MoELayer:
    """A mixture-of-experts layer from router logits to token outputs around an `ExpertMLP`.

    forward(x, logits): route, dispatch with the weights as the rows' scales (the activation applies
    them), the expert MLP with device-resident split sizes, combine.  backward(dy) returns the MLP's
    gradients plus `dx` and `dlogits`; with the MLP's delay_wgrad its backward_dw() is still to be called.
    Row buffers are allocated for each step, tokens * topk rows each, so that a captured step keeps its
    own; rows behind the last used one are neither read nor written.
    """

    def __init__(self, mlp, topk, score="softmax", renormalize=True, scale=1.0):
        self.mlp, self.topk = mlp, int(topk)
        self.route = dict(score=score, renormalize=renormalize, scale=scale)
        self.ctx = None

    def forward(self, x, logits):
        """x [tokens, hidden] BF16, logits [tokens, experts] BF16 or FP32 -> y [tokens, hidden] BF16."""
        _check("x", x, (torch.bfloat16,), 2, contiguous=False)
        _check("logits", logits, _FLOATS, 2, x.device, contiguous=False)
        _shape("logits", logits, (x.shape[0], self.mlp.e))
        _shape("x", x, (x.shape[0], self.mlp.h))
        if x.shape[0] == 0:
            _fail("x has no tokens")
        cap = x.shape[0] * self.topk
        with torch.cuda.device(x.device):
            idx, w = moe_route(logits, self.topk, **self.route)
            rows = torch.empty((cap, self.mlp.h), dtype=torch.bfloat16, device=x.device)
            probs = torch.empty(cap, dtype=torch.float32, device=x.device)
            groups = N.DeviceGroups(self.mlp.e, cap, device=x.device)
            row, _ = moe_dispatch(idx, self.mlp.e, x, rows, weights=w, row_weights=probs, split_sizes=groups.splits)
            y = moe_combine(row, self.mlp.forward(rows, probs, groups))
        self.ctx = dict(logits=logits, idx=idx, row=row)
        return y

    def backward(self, dy):
        """Gradients: the MLP's, with its row gradients replaced by `dx` [tokens, hidden] and `dlogits`."""
        c = self.ctx
        if c is None:
            _fail("backward() without a forward")
        row = c["row"]
        _shape("dy", _check("dy", dy, (torch.bfloat16,), 2, row.device, contiguous=False), (row.shape[0], self.mlp.h))
        self.ctx = None
        with torch.cuda.device(dy.device):
            drows = torch.empty((row.numel(), self.mlp.h), dtype=torch.bfloat16, device=dy.device)
            moe_combine_bwd(row, dy, drows)
            grads = self.mlp.backward(drows)
            dx_rows, dprobs = grads.pop("dx1", None), grads.pop("dprobs", None)
            dw = None
            if dx_rows is not None:
                grads["dx"], dw = moe_dispatch_bwd(row, dx_rows, drow_weights=dprobs)
            elif dprobs is not None:
                # the tokens need no gradient: every slot fetches its row's scale gradient
                dw, _ = moe_dispatch_bwd(row.view(-1, 1), dprobs.view(-1, 1))
                dw = dw.view(row.shape)
            if dw is not None:
                grads["dlogits"] = moe_route_bwd(c["logits"], c["idx"], dw, **self.route)
        return grads
