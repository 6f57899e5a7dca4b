"""Training of the shared (always-on, bf16) experts: the forward that keeps the
pre-activations, its backward, and both as one torch autograd function.

Tensors are torch device tensors, contiguous, all on one device; the work is
enqueued on that device's current stream (or `stream`).  Every computation
happens in libk3moe's kernels; this file only marshals."""
from functools import lru_cache

import torch

from . import (BF16, F32, FMT_BF16, OP_SHARED_BACKWARD, OP_SHARED_TRAIN, check_workspace,
               current_stream, k3moe_shared_ffn_backward, k3moe_shared_ffn_train,
               k3moe_workspace_bytes, make_bank, make_shape, on_device)

_DT = {torch.float32: F32, torch.bfloat16: BF16}


def _need(t, name, shape, device):
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} is {t.dtype}; torch.bfloat16 is needed")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; {tuple(shape)} is needed")
    if t.device != device or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on the weights' GPU")


@lru_cache(maxsize=256)
def _shape_of(T, d, fs, S, out_dtype, op):
    # the routed part of the shape is not used by these calls
    shape = make_shape(T, d, 32, 1, 1, S, fs, BF16, _DT[out_dtype])
    return shape, max(k3moe_workspace_bytes(shape, op), 256)


def _problem(x, w13, w2, out_dtype, op):
    if w13.dim() != 3 or w13.shape[1] % 2 or x.dim() != 2:
        raise ValueError(f"w13 {tuple(w13.shape)} is [S][2 fs][d] and x {tuple(x.shape)} is [T][d]")
    S, two_fs, d = w13.shape
    fs, T, dev = two_fs // 2, x.shape[0], w13.device
    if out_dtype not in _DT:
        raise TypeError(f"y is float32 or bfloat16, not {out_dtype}")
    _need(x, "x", (T, d), dev)
    _need(w13, "w13", (S, two_fs, d), dev)
    _need(w2, "w2", (S, d, fs), dev)
    shape, nbytes = _shape_of(T, d, fs, S, out_dtype, op)
    return shape, make_bank(FMT_BF16, S, d, fs, w13, None, w2, None), nbytes, (T, d, fs, S, dev)


def shared_ffn_train(x, w13, w2, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """y [T][d] = sum over the experts of W2 (silu(Wg x) * (Wu x)) and gu
    [T][S][2 fs], the pre-activations that shared_ffn_backward takes.
    x [T][d], w13 [S][2 fs][d] (gate rows, then up rows), w2 [S][d][fs], bf16."""
    shape, bank, nbytes, (T, d, fs, S, dev) = _problem(x, w13, w2, out_dtype, OP_SHARED_TRAIN)
    with on_device(dev, stream):
        y = torch.empty((T, d), dtype=out_dtype, device=dev)
        gu = torch.empty((T, S, 2 * fs), dtype=torch.bfloat16, device=dev)
        if T:
            if workspace is None:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            else:
                check_workspace(workspace, dev.index)
            k3moe_shared_ffn_train(shape, bank, x, gu, y, workspace, current_stream(dev))
    return y, gu


def shared_ffn_backward(x, gu, dy, w13, w2, need=(True, True, True), workspace=None, stream=None):
    """dx [T][d], dw13 [S][2 fs][d], dw2 [S][d][fs] (bf16) from dy [T][d] bf16 and
    the forward's x and gu; None in the place of one that `need` leaves out."""
    shape, bank, nbytes, (T, d, fs, S, dev) = _problem(x, w13, w2, torch.bfloat16,
                                                       OP_SHARED_BACKWARD)
    _need(gu, "gu", (T, S, 2 * fs), dev)
    _need(dy, "dy", (T, d), dev)
    with on_device(dev, stream):
        dx = torch.empty_like(x) if need[0] else None
        dw13 = torch.empty_like(w13) if need[1] else None
        dw2 = torch.empty_like(w2) if need[2] else None
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        else:
            check_workspace(workspace, dev.index)
        # (an empty tensor's address may be NULL: for T = 0 nothing is read or written there)
        k3moe_shared_ffn_backward(shape, bank, x, gu, dy, dx if T else None, dw13, dw2, workspace,
                                  current_stream(dev))
    return dx, dw13, dw2


class _SharedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w13, w2):
        y, gu = shared_ffn_train(x, w13, w2)
        ctx.save_for_backward(x, gu, w13, w2)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, gu, w13, w2 = ctx.saved_tensors
        return shared_ffn_backward(x, gu, dy.contiguous(), w13, w2, need=ctx.needs_input_grad)


def shared_ffn(x, w13, w2):
    """The shared experts as a torch operation: y [T][d] bf16, differentiable once
    in x, w13 and w2.  Capture its backward together with its forward, with no eager
    graph of the same leaves alive (torch accumulates their gradients on the stream
    that graph was recorded on), or capture the two halves above."""
    return _SharedFFN.apply(x, w13, w2)
