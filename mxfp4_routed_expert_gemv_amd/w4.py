"""Products with 4-bit integer weights and group scales (k3moe_w4_linear,
k3moe_w4_glu) on torch tensors.  Every computation happens in libk3moe's
kernels; this file only marshals."""
import ctypes

import torch
from torch.autograd.graph import increment_version

from . import BF16, F32, K3moeError, W4Matrix, check_workspace, lib, on_device

_U8, _BF16 = torch.uint8, torch.bfloat16
_raw_stream = torch._C._cuda_getCurrentRawStream
_DT = {torch.float32: F32, torch.bfloat16: BF16}


def _run(call, half, x, codes, scale, zero, out_dtype, out, workspace, stream):
    try:
        (n, half_k), (T, k), (rows, groups) = codes.shape, x.shape, scale.shape
    except ValueError:
        n = half_k = T = k = rows = groups = 0
    if 2 * half_k != k or rows != n or groups < 1 or k % groups:
        raise ValueError(f"x {tuple(x.shape)}, codes {tuple(codes.shape)} and scale "
                         f"{tuple(scale.shape)} are not [T][k], [n][k / 2] and [n][k / group]")
    x_dtype = _DT.get(x.dtype)
    if codes.dtype != _U8 or scale.dtype != _BF16 or x_dtype is None:
        raise TypeError(f"codes {codes.dtype}, scale {scale.dtype} and x {x.dtype} must be uint8, "
                        "bfloat16, and bfloat16 or float32")
    if zero is not None and (zero.dtype != _U8 or zero.shape != scale.shape):
        raise TypeError(f"zero must be uint8 of scale's shape {tuple(scale.shape)}")
    cols = n // 2 if half else n
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    o_dtype = _DT.get(out_dtype)
    if o_dtype is None:
        raise TypeError(f"the output is float32 or bfloat16, not {out_dtype}")
    if out is not None and (out.shape != (T, cols) or out.dtype != out_dtype):
        raise ValueError(f"out must be {(T, cols)} {out_dtype}")
    index = x.get_device()
    if index < 0 or codes.get_device() != index or scale.get_device() != index or not (
            x.is_contiguous() and codes.is_contiguous() and scale.is_contiguous()) or \
            not (zero is None or (zero.get_device() == index and zero.is_contiguous())) or \
            not (out is None or (out.get_device() == index and out.is_contiguous())):
        raise ValueError("the tensors must be contiguous and on one GPU")
    given = out
    w = W4Matrix(n, k, k // groups, codes.data_ptr(), scale.data_ptr(),
                 None if zero is None else zero.data_ptr())
    if stream is None and torch.cuda.current_device() == index:
        status, out = _launch(call, w, T, cols, x, x_dtype, out, out_dtype, o_dtype, workspace, index)
    else:
        with on_device(x.device, stream):
            status, out = _launch(call, w, T, cols, x, x_dtype, out, out_dtype, o_dtype, workspace,
                                  index)
    if status:
        raise K3moeError(status, lib.k3moe_last_error().decode())
    if given is not None:   # autograd has to know what was overwritten
        increment_version(given)
    return out


def _launch(call, w, T, cols, x, x_dtype, out, out_dtype, o_dtype, ws, index):
    if out is None:
        out = torch.empty((T, cols), dtype=out_dtype, device=x.device)
    if T <= 16:
        wp, wb = None, 0
    else:
        if ws is None:
            ws = torch.empty(lib.k3moe_w4_workspace_bytes(ctypes.byref(w), T), dtype=_U8,
                             device=x.device)
        else:
            check_workspace(ws, index)
        wp, wb = ws.data_ptr(), ws.numel() * ws.element_size()
    return call(ctypes.byref(w), T, x_dtype, o_dtype, x.data_ptr(), out.data_ptr(), wp, wb,
                _raw_stream(index)), out


def w4_linear(x, codes, scale, zero=None, out_dtype=None, out=None, workspace=None, stream=None):
    """out [T][n] = x W^T with W[r][j] = (q[r][j] - zero[r][j / g]) * scale[r][j / g]:
    x [T][k] (bf16 or fp32), codes [n][k / 2] uint8 (low nibble = even element),
    scale [n][k / g] bf16, zero [n][k / g] uint8 (None: 8 everywhere).
    out_dtype: bf16 or fp32, x's by default.  workspace: a uint8 tensor of
    k3moe_w4_workspace_bytes (made when needed, above 16 tokens, if not given).
    The result carries no gradient."""
    return _run(lib.k3moe_w4_linear, False, x, codes, scale, zero, out_dtype, out, workspace, stream)


def w4_glu(x, codes, scale, zero=None, out_dtype=None, out=None, workspace=None, stream=None):
    """The gated block's first half, silu(x Wg^T) * (x Wu^T) [T][n / 2]: the first
    n / 2 rows of W are the gate, the others the up projection."""
    return _run(lib.k3moe_w4_glu, True, x, codes, scale, zero, out_dtype, out, workspace, stream)
