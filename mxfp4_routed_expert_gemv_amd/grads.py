"""The global gradient norm and clipping (k3moe_grad_norm, k3moe_grad_clip) on
lists of torch tensors.  Every computation happens in libk3moe's kernels; this
file only marshals."""
from array import array

import torch

from . import BF16, F32, k3moe_grad_clip, k3moe_grad_norm, k3moe_grad_workspace_bytes

_DT = {torch.float32: F32, torch.bfloat16: BF16}


def _table(tensors, outs):
    """The k3moe_tensor list: four words a tensor, the two types in the last."""
    dev = tensors[0].device
    try:
        words = array("q")
        for t, o in zip(tensors, outs):
            words.extend((t.data_ptr(), o.data_ptr(), t.numel(), _DT[t.dtype] | _DT[o.dtype] << 32))
            if t.device != dev or o.device != dev or not (t.is_contiguous() and o.is_contiguous()):
                raise ValueError("the tensors must be contiguous and on one device")
            if o.shape != t.shape:
                raise ValueError(f"an output of shape {tuple(o.shape)} for {tuple(t.shape)}")
    except KeyError as e:
        raise TypeError(f"gradients are float32 or bfloat16, not {e.args[0]}") from None
    return words, dev


def _call(run, tensors, outs, stream):
    tensors = list(tensors)
    outs = tensors if outs is None else list(outs)
    if not tensors:
        raise ValueError("no tensors")
    if len(outs) != len(tensors):
        raise ValueError(f"{len(outs)} outputs for {len(tensors)} tensors")
    words, dev = _table(tensors, outs)
    n = len(tensors)
    with torch.cuda.device(dev):
        norm = torch.empty((), dtype=torch.float32, device=dev)
        ws = torch.empty(k3moe_grad_workspace_bytes(n), dtype=torch.uint8, device=dev)
        run(words.buffer_info()[0], n, norm, ws, stream)
    return norm


def grad_norm(tensors, stream=None):
    """The 2-norm over all elements of all tensors (fp32 or bf16, contiguous, on
    one device), a device fp32 scalar; the host does not wait."""
    return _call(k3moe_grad_norm, tensors, None, stream)


def clip_grads(tensors, max_norm, out=None, stream=None):
    """Scales the tensors by min(1, max_norm / norm), in place or into the tensors
    `out` (fp32 or bf16 each, of the same shapes), and returns the norm as
    grad_norm does.  A norm that is not finite scales nothing."""
    return _call(lambda ts, n, norm, ws, st: k3moe_grad_clip(ts, n, float(max_norm), norm, ws, st),
                 tensors, out, stream)
