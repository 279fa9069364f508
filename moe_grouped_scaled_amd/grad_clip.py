"""The global norm of many gradients, and clipping by it.

Both enqueue the library's kernels on the tensors' device, on its current stream (or on `stream`, as in `moe`), and
return the norm as an FP32 scalar tensor on that device: nothing synchronises, and a captured step clips by each
replay's own norm.  The addresses of the gradients travel with the call.
"""

import array

import torch

from . import _native as N
from .moe import _call, _fail, _on_stream

_TYPES = {torch.bfloat16: 0, torch.float32: 1}


def _tensor(what, t, device):
    if not isinstance(t, torch.Tensor):
        _fail("%s must be a tensor", what)
    if t.dtype not in _TYPES:
        _fail("%s has type %s, expected torch.bfloat16 or torch.float32", what, t.dtype)
    if not t.is_contiguous():
        _fail("%s must be contiguous", what)
    if not t.is_cuda:
        _fail("%s must be on a GPU", what)
    if device is not None and t.device != device:
        _fail("%s is on %s, expected %s", what, t.device, device)
    return t


def _run(grads, clip, max_norm, eps, out, workspace, norm):
    if not grads:
        _fail("grads is empty")
    if out is not None and len(out) != len(grads):
        _fail("out has %d tensors, grads has %d", len(out), len(grads))
    dev = _tensor("grads[0]", grads[0], None).device
    # mgs_grad rows: address, output's address, elements, the two types in one word
    rows, index, types, is_tensor = [], dev.index, _TYPES, torch.Tensor
    for i, g in enumerate(grads):
        o = g if out is None else out[i]
        t, u = (types.get(g.dtype), types.get(o.dtype)) if isinstance(g, is_tensor) and isinstance(o, is_tensor) else (None, None)
        if (t is None or u is None or g.get_device() != index or o.get_device() != index
                or not (g.is_contiguous() and o.is_contiguous())):
            _tensor("grads[%d]" % i, g, dev)
            _tensor("out[%d]" % i, o, dev)
        n = g.numel()
        if o is g:
            at = g.data_ptr()
            rows += (at, at, n, t << 32 | t)
            continue
        if o.numel() != n:
            _fail("out[%d] has %d elements, expected %d", i, o.numel(), n)
        rows += (g.data_ptr(), o.data_ptr(), n, u << 32 | t)
    table = array.array("q", rows)
    at = table.buffer_info()[0]
    need = N.LIB.mgs_grad_norm_workspace_bytes(len(grads), at)
    if need < 0:
        N._check(int(need))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        _fail("workspace must be contiguous and on %s", dev)
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=dev)
    elif norm.dtype != torch.float32 or norm.numel() != 1 or norm.device != dev:
        _fail("norm must be one FP32 element on %s", dev)
    _call(dev, N.LIB.mgs_grad_norm, len(grads), at, norm.data_ptr(), workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), int(clip), float(max_norm), float(eps))
    return norm


def grad_norm(grads, norm=None, workspace=None, stream=None):
    """The 2-norm of all elements of all `grads` (BF16 or FP32, contiguous, of any sizes), summed in 64 bits."""
    grads = list(grads)
    if stream is not None:
        return _on_stream(stream, grads[0] if grads else None, grad_norm, grads, norm, workspace)
    return _run(grads, False, 0.0, 0.0, None, workspace, norm)


def clip_grad_norm(grads, max_norm, eps=1e-6, out=None, norm=None, workspace=None, stream=None):
    """Scales `grads` by min(1, max_norm / (norm + eps)), in place or into `out` (contiguous tensors of as many elements,
    BF16 or FP32), and returns the norm before that.  A NaN norm makes every result NaN, an infinite gradient zeros (NaN in its
    own place); a finite norm past FP32's range is returned as infinity and clips like any other."""
    grads = list(grads)
    if stream is not None:
        return _on_stream(stream, grads[0] if grads else None, clip_grad_norm, grads, max_norm, eps, out, norm, workspace)
    return _run(grads, True, max_norm, eps, None if out is None else list(out), workspace, norm)
