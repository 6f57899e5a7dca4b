"""The global gradient norm and clipping (k3moe_grad_norm, k3moe_grad_clip) on
lists of torch tensors.  Every computation happens in libk3moe's kernels; this
file only marshals."""
from itertools import chain
from operator import attrgetter
from struct import pack

import torch
from torch.autograd.graph import increment_version

from . import (BF16, F32, current_stream, k3moe_grad_clip, k3moe_grad_norm,
               k3moe_grad_workspace_bytes, on_device)

_DT = {torch.float32: F32, torch.bfloat16: BF16}
_dtype, _shape, _T = attrgetter("dtype"), attrgetter("shape"), torch.Tensor


def _types(tensors):
    types = list(map(_DT.get, map(_dtype, tensors)))
    if None in types:
        raise TypeError("gradients are float32 or bfloat16, not "
                        f"{tensors[types.index(None)].dtype}")
    return types


def _call(run, tensors, outs, stream, clip):
    tensors = list(tensors)
    if not tensors:
        raise ValueError("no tensors")
    dev = tensors[0].device
    every = tensors
    types = _types(tensors)
    pointers = to = list(map(_T.data_ptr, tensors))
    if outs is not None:
        outs = list(outs)
        if len(outs) != len(tensors):
            raise ValueError(f"{len(outs)} outputs for {len(tensors)} tensors")
        if list(map(_shape, outs)) != list(map(_shape, tensors)):
            raise ValueError("the outputs' shapes are not the tensors'")
        every = tensors + outs
        to = list(map(_T.data_ptr, outs))
        types = [t | o << 32 for t, o in zip(types, _types(outs))]
    else:
        types = [t | t << 32 for t in types]
    if dev.type != "cuda" or set(map(_T.get_device, every)) != {dev.index} or \
            not all(map(_T.is_contiguous, every)):
        raise ValueError("the tensors must be contiguous and on one device")
    # the k3moe_tensor list: four words a tensor, the two types in the last
    n = len(tensors)
    words = pack(f"{4 * n}q", *chain.from_iterable(zip(pointers, to, map(_T.numel, tensors), types)))
    with on_device(dev, stream):
        norm = torch.empty((), dtype=torch.float32, device=dev)
        ws = torch.empty(k3moe_grad_workspace_bytes(n), dtype=torch.uint8, device=dev)
        run(words, n, norm, ws, current_stream(dev))
    if clip:   # autograd has to know what was overwritten
        increment_version(outs or tensors)
    return norm


def grad_norm(tensors, stream=None):
    """The 2-norm over all elements of all tensors (fp32 or bf16, contiguous, on
    one device), a device fp32 scalar; the host does not wait."""
    return _call(k3moe_grad_norm, tensors, None, stream, False)


def clip_grads(tensors, max_norm, out=None, stream=None):
    """Scales the tensors by min(1, max_norm / norm), in place or into the tensors
    `out` (fp32 or bf16 each, of the same shapes), and returns the norm as
    grad_norm does.  A norm of infinities or NaN scales nothing."""
    return _call(lambda ts, n, norm, ws, st: k3moe_grad_clip(ts, n, float(max_norm), norm, ws, st),
                 tensors, out, stream, True)
