"""Routing around the expert MLP: router, dispatch into expert order, combine, their gradients, and the layer.

The functions check their tensors, allocate the outputs that are not given and enqueue the library's
kernels on the tensors' device, on its current stream.  With `stream` (a torch.cuda.Stream of that device
or a HIP stream handle, 0 the null stream) they do as under ``torch.cuda.stream(stream)``: what they allocate
belongs to that stream too.  Nothing synchronises: the split sizes stay in device memory, where
`_native.DeviceGroups` takes them, so a captured graph follows the routing.  An output must not be or overlap
another tensor of the call.

A slot is one (token, choice) pair, numbered token * topk + choice; a slot without an expert has expert -1
and row -1.
"""

import torch

from . import _native as N


def _fail(msg, *args):
    raise ValueError(msg % args if args else msg)


def _check(what, t, dtypes, ndim, device=None, contiguous=True, shape=None):
    """A CUDA tensor of one of `dtypes`, `ndim` dimensions and unit column stride (rows contiguous when
    `contiguous`), on `device`, of `shape`."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.is_cuda and (device is None or t.device == device)
            and (t.dim() == ndim if shape is None else t.shape == shape) and t.is_contiguous()):
        return t
    if not isinstance(t, torch.Tensor):
        _fail("%s must be a tensor", what)
    if t.dtype not in dtypes:
        _fail("%s has type %s, expected %s", what, t.dtype, " or ".join(str(d) for d in dtypes))
    if t.dim() != ndim:
        _fail("%s has %d dimensions, expected %d", what, t.dim(), ndim)
    if shape is not None and tuple(t.shape) != tuple(shape):
        _fail("%s has shape %s, expected %s", what, tuple(t.shape), tuple(shape))
    if not t.is_contiguous():
        if contiguous:
            _fail("%s must be contiguous", what)
        if t.numel() and (t.stride(1) != 1 and t.shape[1] > 1 or t.stride(0) < t.shape[1] and t.shape[0] > 1):
            _fail("%s must have unit column stride and rows that do not overlap (strides %s)", what, t.stride())
    if not t.is_cuda:
        _fail("%s must be on a GPU", what)
    if device is not None and t.device != device:
        _fail("%s is on %s, expected %s", what, t.device, device)
    return t


def _ld(t):
    """Row stride in elements (a single row may carry any stride)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _call(device, fn, *args):
    """fn(*args, stream handle) with the tensors' device current, its error raised."""
    index = device.index
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc:
        N._check(rc)


def _on_stream(stream, t, fn, *args):
    """fn(*args) with `stream` current; `t` is one of its tensors."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return fn(*args)  # refused there
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, t.device) if stream else torch.cuda.default_stream(t.device)
    if stream.device != t.device:
        _fail("the stream is on %s, the tensors are on %s", stream.device, t.device)
    with torch.cuda.stream(stream):
        return fn(*args)


def _int32(what, n):
    """(The binding passes 32-bit arguments on without their upper bits; the library checks the rest.)"""
    if n >> 31:
        _fail("%s = %d is out of range", what, n)


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
    if stream is not None:
        return _on_stream(stream, logits, moe_route, logits, topk, score, renormalize, scale, expert_idx, weights)
    _int32("topk", topk)
    _check("logits", logits, _FLOATS, 2, contiguous=False)
    t, e = logits.shape
    dev = logits.device
    if expert_idx is None:
        expert_idx = torch.empty((t, topk), dtype=torch.int32, device=dev)
    else:
        _check("expert_idx", expert_idx, _I32, 2, dev, shape=(t, topk))
    if weights is None:
        weights = torch.empty((t, topk), dtype=torch.float32, device=dev)
    else:
        _check("weights", weights, _F32, 2, dev, shape=(t, topk))
    _call(dev, N.LIB.mgs_moe_route, _params(score, renormalize, scale), t, e, topk, logits.data_ptr(),
          N.DTYPE[logits.dtype], _ld(logits), expert_idx.data_ptr(), weights.data_ptr())
    return expert_idx, weights


def moe_route_bwd(logits, expert_idx, dweights, score="softmax", renormalize=True, scale=1.0, dlogits=None, stream=None):
    """The logits' gradient of `moe_route`'s weights (every element of dlogits is written)."""
    if stream is not None:
        return _on_stream(stream, logits, moe_route_bwd, logits, expert_idx, dweights, score, renormalize, scale, dlogits)
    _check("logits", logits, _FLOATS, 2, contiguous=False)
    t, e = logits.shape
    dev = logits.device
    _check("expert_idx", expert_idx, _I32, 2, dev)
    k = expert_idx.shape[1]
    if expert_idx.shape[0] != t:
        _fail("expert_idx has %d rows, expected %d", expert_idx.shape[0], t)
    _check("dweights", dweights, _F32, 2, dev, shape=(t, k))
    if dlogits is None:
        dlogits = logits.new_empty((t, e))
    else:
        _check("dlogits", dlogits, (logits.dtype,), 2, dev, contiguous=False, shape=(t, e))
    _call(dev, N.LIB.mgs_moe_route_bwd, _params(score, renormalize, scale), t, e, k, logits.data_ptr(),
          N.DTYPE[logits.dtype], _ld(logits), expert_idx.data_ptr(), dweights.data_ptr(), dlogits.data_ptr(), _ld(dlogits))
    return dlogits


def moe_dispatch_workspace_bytes(tokens, topk, num_experts):
    _int32("topk", topk)
    _int32("num_experts", num_experts)
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
    if stream is not None:
        return _on_stream(stream, expert_idx, moe_dispatch, expert_idx, num_experts, x, rows, weights, row_weights, row_of_slot, split_sizes,
                          workspace)
    _int32("num_experts", num_experts)
    _check("expert_idx", expert_idx, _I32, 2)
    t, k = expert_idx.shape
    dev = expert_idx.device
    need = moe_dispatch_workspace_bytes(t, k, num_experts)
    if row_of_slot is None:
        row_of_slot = torch.empty_like(expert_idx)
    else:
        _check("row_of_slot", row_of_slot, _I32, 2, dev, shape=(t, k))
    if split_sizes is None:
        split_sizes = torch.empty(num_experts, dtype=torch.int64, device=dev)
    else:
        _check("split_sizes", split_sizes, _I64, 1, dev, shape=(num_experts,))
    ws, wb = None, 0
    if need:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        ws, wb = _check("workspace", workspace, (torch.uint8,), 1, dev).data_ptr(), workspace.numel()
    h, dt, ldx, xp, rp, n, wp, rwp = 0, 0, 0, None, None, 0, None, None
    if x is not None or rows is not None or weights is not None or row_weights is not None:
        if x is None or rows is None:
            _fail("x and rows go together (and weights need them)")
        _check("x", x, _FLOATS, 2, dev, contiguous=False)
        h, n = x.shape[1], rows.shape[0]
        if x.shape[0] != t:
            _fail("x has %d rows, expected %d", x.shape[0], t)
        _check("rows", rows, (x.dtype,), 2, dev, shape=(n, h))
        dt, ldx, xp, rp = N.DTYPE[x.dtype], _ld(x), x.data_ptr(), rows.data_ptr()
        if (weights is None) != (row_weights is None):
            _fail("weights and row_weights go together")
        if weights is not None:
            wp = _check("weights", weights, _F32, 2, dev, shape=(t, k)).data_ptr()
            rwp = _check("row_weights", row_weights, _F32, 1, dev, shape=(n,)).data_ptr()
    _call(dev, N.LIB.mgs_moe_dispatch, t, k, num_experts, expert_idx.data_ptr(), h, dt, xp, ldx, wp, rp, n, rwp,
          row_of_slot.data_ptr(), split_sizes.data_ptr(), ws, wb)
    return row_of_slot, split_sizes


def _slots_and_rows(row_of_slot, rows, name="rows"):
    _check("row_of_slot", row_of_slot, _I32, 2)
    _check(name, rows, _FLOATS, 2, row_of_slot.device)
    return row_of_slot.shape[0], row_of_slot.shape[1], rows.shape[1], rows.shape[0], row_of_slot.device


def moe_dispatch_bwd(row_of_slot, drows, drow_weights=None, dx=None, dweights=None, stream=None):
    """Gradient of the dispatch: dx[t] = the sum of the token's drows, and with `drow_weights` (FP32, one a row)
    dweights[t, c] = drow_weights[row_of_slot[t, c]].  Returns (dx, dweights or None)."""
    if stream is not None:
        return _on_stream(stream, row_of_slot, moe_dispatch_bwd, row_of_slot, drows, drow_weights, dx, dweights)
    t, k, h, n, dev = _slots_and_rows(row_of_slot, drows, "drows")
    if dx is None:
        dx = drows.new_empty((t, h))
    else:
        _check("dx", dx, (drows.dtype,), 2, dev, contiguous=False, shape=(t, h))
    dwp = gwp = None
    if drow_weights is not None:
        gwp = _check("drow_weights", drow_weights, _F32, 1, dev, shape=(n,)).data_ptr()
        if dweights is None:
            dweights = drow_weights.new_empty((t, k))
        dwp = _check("dweights", dweights, _F32, 2, dev, shape=(t, k)).data_ptr()
    elif dweights is not None:
        _fail("dweights needs drow_weights")
    _call(dev, N.LIB.mgs_moe_dispatch_bwd, t, k, h, N.DTYPE[drows.dtype], row_of_slot.data_ptr(), n,
          drows.data_ptr(), gwp, dx.data_ptr(), _ld(dx), dwp)
    return dx, dweights


def moe_combine(row_of_slot, rows, weights=None, y=None, stream=None):
    """y[t] = the sum over the token's slots of weights[t, c] * rows[row_of_slot[t, c]] (weights 1 when None),
    in FP32 with one rounding."""
    if stream is not None:
        return _on_stream(stream, row_of_slot, moe_combine, row_of_slot, rows, weights, y)
    t, k, h, n, dev = _slots_and_rows(row_of_slot, rows)
    if y is None:
        y = rows.new_empty((t, h))
    else:
        _check("y", y, (rows.dtype,), 2, dev, contiguous=False, shape=(t, h))
    wp = None if weights is None else _check("weights", weights, _F32, 2, dev, shape=(t, k)).data_ptr()
    _call(dev, N.LIB.mgs_moe_combine, t, k, h, N.DTYPE[rows.dtype], row_of_slot.data_ptr(), n, rows.data_ptr(), wp,
          y.data_ptr(), _ld(y))
    return y


def moe_combine_bwd(row_of_slot, dy, drows=None, rows=None, weights=None, dweights=None, stream=None):
    """Gradient of the combine: drows[row_of_slot[t, c]] = weights[t, c] * dy[t] (rows no slot has stay as they
    are), and with `rows`, the forward's input, dweights[t, c] = <dy[t], rows[row_of_slot[t, c]]>, which is
    returned (else None)."""
    if stream is not None:
        return _on_stream(stream, row_of_slot, moe_combine_bwd, row_of_slot, dy, drows, rows, weights, dweights)
    _check("row_of_slot", row_of_slot, _I32, 2)
    dev = row_of_slot.device
    t, k = row_of_slot.shape
    _check("dy", dy, _FLOATS, 2, dev, contiguous=False)
    h = dy.shape[1]
    if dy.shape[0] != t:
        _fail("dy has %d rows, expected %d", dy.shape[0], t)
    if drows is None and rows is None:
        _fail("drows or rows is needed")
    n = (rows if drows is None else drows).shape[0]
    rp = None if rows is None else _check("rows", rows, (dy.dtype,), 2, dev, shape=(n, h)).data_ptr()
    dp = None if drows is None else _check("drows", drows, (dy.dtype,), 2, dev, shape=(n, h)).data_ptr()
    wp = None if weights is None else _check("weights", weights, _F32, 2, dev, shape=(t, k)).data_ptr()
    if rows is not None and dweights is None:
        dweights = torch.empty((t, k), dtype=torch.float32, device=dev)
    dwp = None if dweights is None else _check("dweights", dweights, _F32, 2, dev, shape=(t, k)).data_ptr()
    _call(dev, N.LIB.mgs_moe_combine_bwd, t, k, h, N.DTYPE[dy.dtype], row_of_slot.data_ptr(), n, dy.data_ptr(),
          _ld(dy), rp, wp, dp, dwp)
    return dweights


class MoELayer:
    """A mixture-of-experts layer from router logits to token outputs around an `ExpertMLP`.

    forward(x, logits): y[t] = the sum over the token's experts of weight * expert(x[t]): route, dispatch, the
    expert MLP with device-resident split sizes, combine.  Without an FC2 bias the weights go with the rows as
    their scales (the activation applies them, FC2 is linear behind it).  With one they are applied by the
    combine, so that they reach the bias too: the rows' scales are 1, and the expert outputs are kept for the
    weights' gradient.  backward(dy) returns the MLP's gradients plus `dx` and `dlogits` (the latter with the
    MLP's grad_probs); with the MLP's delay_wgrad its backward_dw() is still to be called.
    Row buffers are allocated for each step, tokens * topk rows each, so that a captured step keeps its
    own; rows behind the last used one are neither read nor written.  Without tokens (x [0, hidden]) the outputs
    are empty and the weights' gradients zeros.  The MLP keeps one forward's tensors at a time, so layers that
    share one alternate forward and backward; a backward whose forward it no longer holds is refused.
    """

    def __init__(self, mlp, topk, score="softmax", renormalize=True, scale=1.0):
        self.mlp, self.topk = mlp, int(topk)
        self.route = dict(score=score, renormalize=renormalize, scale=scale)
        self.ctx = None

    def forward(self, x, logits):
        """x [tokens, hidden] BF16, logits [tokens, experts] BF16 or FP32 -> y [tokens, hidden] BF16."""
        _check("x", x, (torch.bfloat16,), 2, contiguous=False)
        _check("x", x, (torch.bfloat16,), 2, contiguous=False, shape=(x.shape[0], self.mlp.h))
        _check("logits", logits, _FLOATS, 2, x.device, contiguous=False, shape=(x.shape[0], self.mlp.e))
        for t in (self.mlp.w1, self.mlp.w2, self.mlp.b1, self.mlp.b2):
            if t is not None and t.device != x.device:
                _fail("x is on %s, the expert MLP's parameters are on %s", x.device, t.device)
        cap = max(x.shape[0] * self.topk, 1)  # (without tokens: buffers of one row that nothing uses)
        with torch.cuda.device(x.device):
            idx, w = moe_route(logits, self.topk, **self.route)
            rows = torch.empty((cap, self.mlp.h), dtype=torch.bfloat16, device=x.device)
            groups = N.DeviceGroups(self.mlp.e, cap, device=x.device)
            ctx = dict(logits=logits, idx=idx)
            if self.mlp.b2 is None:
                probs = torch.empty(cap, dtype=torch.float32, device=x.device)
                row, _ = moe_dispatch(idx, self.mlp.e, x, rows, weights=w, row_weights=probs, split_sizes=groups.splits)
                y = moe_combine(row, self.mlp.forward(rows, probs, groups))
            else:
                probs = torch.ones(cap, dtype=torch.float32, device=x.device)
                row, _ = moe_dispatch(idx, self.mlp.e, x, rows, split_sizes=groups.splits)
                y_rows = self.mlp.forward(rows, probs, groups)
                y = moe_combine(row, y_rows, weights=w)
                ctx.update(w=w, y_rows=y_rows if self.mlp.grad_probs else None)
        # (a mark in what the MLP saved, not a reference to it: that is the MLP's to free)
        mark = self.mlp.ctx["owner"] = object()
        self.ctx = dict(ctx, row=row, cap=cap, mark=mark)
        return y

    def backward(self, dy):
        """Gradients: the MLP's, with its row gradients replaced by `dx` [tokens, hidden] and `dlogits`."""
        c = self.ctx
        if c is None:
            _fail("backward() without a forward")
        row = c["row"]
        _check("dy", dy, (torch.bfloat16,), 2, row.device, contiguous=False, shape=(row.shape[0], self.mlp.h))
        if (self.mlp.ctx or {}).get("owner") is not c["mark"]:
            self.ctx = None
            _fail("the expert MLP has run another forward or its backward since: what this one saved is gone")
        self.ctx = None
        with torch.cuda.device(dy.device):
            drows = torch.empty((c["cap"], self.mlp.h), dtype=torch.bfloat16, device=dy.device)
            if "w" in c:  # the combine's weights
                dw = moe_combine_bwd(row, dy, drows, rows=c["y_rows"], weights=c["w"])
            else:
                dw = moe_combine_bwd(row, dy, drows)
            grads = self.mlp.backward(drows)
            dx_rows, dprobs = grads.pop("dx1", None), grads.pop("dprobs", None)
            if "w" in c:
                dprobs = None  # of the rows' scales of 1
            if dx_rows is not None:
                grads["dx"], got = moe_dispatch_bwd(row, dx_rows, drow_weights=dprobs)
                dw = got if dw is None else dw
            elif dprobs is not None:
                # the tokens need no gradient: every slot fetches its row's scale gradient
                dw, _ = moe_dispatch_bwd(row.view(-1, 1), dprobs.view(-1, 1))
                dw = dw.view(row.shape)
            if dw is not None:
                grads["dlogits"] = moe_route_bwd(c["logits"], c["idx"], dw, **self.route)
        return grads
