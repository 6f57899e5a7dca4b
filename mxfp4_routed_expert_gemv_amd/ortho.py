"""The orthogonalised update of weight matrices (k3moe_orthogonalize) on torch
tensors.  Every computation happens in libk3moe's kernels; this file only
marshals."""
import ctypes
from functools import lru_cache

import torch
from torch.autograd.graph import increment_version

from . import (BF16, F32, Ortho, check_workspace, current_stream, k3moe_orthogonalize,
               k3moe_orthogonalize_workspace_bytes, on_device)

_DT = {torch.float32: F32, torch.bfloat16: BF16}
MUON = (3.4445, -4.7750, 2.0315)   # a, b, c: every singular value to 0.7 .. 1.2 in five steps


@lru_cache(maxsize=256)
def _problem(batch, m, n, dtype, steps, coefficients, scale):
    if len(coefficients) == 3 and not isinstance(coefficients[0], tuple):
        coefficients = (coefficients,) * max(steps, 0)
    if len(coefficients) != steps or any(len(c) != 3 for c in coefficients):
        raise ValueError(f"coefficients are (a, b, c), or one such triple for each of {steps} steps")
    flat = [float(v) for c in coefficients for v in c]
    p = Ortho(batch, m, n, _DT[dtype], steps, (ctypes.c_float * len(flat))(*flat), scale)
    return p, k3moe_orthogonalize_workspace_bytes(p)


def orthogonalize(g, steps=5, coefficients=MUON, scale=1.0, out=None, workspace=None, stream=None):
    """scale times the matrix with g's singular vectors and every singular value
    taken towards 1 by `steps` Newton-Schulz steps X = a X + b (X X^T) X + c (X X^T)^2 X
    from X = g / |g|, in bf16.  g [m][n], or a stack [..][m][n], bf16 or fp32 (a stack
    of no matrices gives none); coefficients: (a, b, c), or such a triple for each step;
    out: a bf16 tensor of g's shape, g itself among them.  The result carries no
    gradient.  Sums are fp32; matrices with a short side over 128 enter the products in
    fp16, which five of MUON's steps end with within 3e-3 of the exact result in norm where
    the singular values are spread, 5e-3 where all are equal (1.7e-3 of it the rounding to
    bf16); smaller ones keep 22 bits."""
    if g.dim() < 2:
        raise ValueError(f"g {tuple(g.shape)} is a matrix or a stack of them")
    if g.dtype not in _DT:
        raise TypeError(f"g is float32 or bfloat16, not {g.dtype}")
    if not g.is_cuda or not g.is_contiguous():
        raise ValueError("g must be a contiguous tensor on a GPU")
    if out is not None:
        if out.dtype != torch.bfloat16:
            raise TypeError(f"out is {out.dtype}; torch.bfloat16 is needed")
        if out.shape != g.shape or out.device != g.device or not out.is_contiguous():
            raise ValueError("out must be a contiguous tensor of g's shape on its GPU")
        a, b = g.data_ptr(), out.data_ptr()
        if a < b + out.nbytes and b < a + g.nbytes and (a != b or g.dtype != out.dtype):
            raise ValueError("out overlaps g, and is not g itself")
    m, n = g.shape[-2:]
    dev, given = g.device, out
    with on_device(dev, stream):
        # the call takes its tensors at 16 bytes: a part of a larger one (a bucket of
        # gradients) that begins elsewhere is copied, and its result too
        if out is None or out.data_ptr() & 15:
            out = torch.empty(g.shape, dtype=torch.bfloat16, device=dev)
        if out.numel() == 0:
            return out if given is None else given
        key = tuple(tuple(c) if hasattr(c, "__len__") else float(c) for c in coefficients)
        p, nbytes = _problem(g.numel() // (m * n), m, n, g.dtype, int(steps), key, float(scale))
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        else:
            check_workspace(workspace, dev.index)
        if g.data_ptr() & 15:
            g = g.clone()
        k3moe_orthogonalize(p, g, out, workspace, current_stream(dev))
        if given is not None and given is not out:
            given.detach().copy_(out)
    if given is None:
        return out
    increment_version(given)   # autograd has to know what was overwritten
    return given
