"""Products with 4-bit integer weights and group scales (k3moe_w4_linear,
k3moe_w4_glu) on torch tensors.  Every computation happens in libk3moe's
kernels; this file only marshals."""
import ctypes

import torch

from . import BF16, F32, K3moeError, W4Matrix, current_stream, lib, on_device

_DT = {torch.float32: F32, torch.bfloat16: BF16}


def _run(call, half, x, codes, scale, zero, out_dtype, out, workspace, stream):
    dev = x.device
    if codes.dim() != 2 or scale.dim() != 2 or x.dim() != 2:
        raise ValueError(f"x {tuple(x.shape)}, codes {tuple(codes.shape)} and scale "
                         f"{tuple(scale.shape)} are [T][k], [n][k / 2] and [n][k / group]")
    (n, bytes_), (T, k), groups = codes.shape, x.shape, scale.shape[1]
    if 2 * bytes_ != k or scale.shape[0] != n or groups < 1 or k % groups:
        raise ValueError(f"x {tuple(x.shape)}, codes {tuple(codes.shape)} and scale "
                         f"{tuple(scale.shape)} do not fit each other")
    if codes.dtype != torch.uint8 or scale.dtype != torch.bfloat16 or x.dtype not in _DT:
        raise TypeError(f"codes {codes.dtype}, scale {scale.dtype} and x {x.dtype} must be uint8, "
                        "bfloat16, and bfloat16 or float32")
    if zero is not None and (zero.dtype != torch.uint8 or zero.shape != scale.shape):
        raise TypeError(f"zero must be uint8 of scale's shape {tuple(scale.shape)}")
    cols = n // 2 if half else n
    if out is None:
        out = torch.empty((T, cols), dtype=x.dtype if out_dtype is None else out_dtype, device=dev)
    elif tuple(out.shape) != (T, cols) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError(f"out must be {(T, cols)} {out_dtype}")
    if out.dtype not in _DT:
        raise TypeError(f"the output is float32 or bfloat16, not {out.dtype}")
    same = dev == codes.device == scale.device == out.device and (zero is None or zero.device == dev)
    if not same or dev.type != "cuda" or not (
            x.is_contiguous() and codes.is_contiguous() and scale.is_contiguous()
            and out.is_contiguous() and (zero is None or zero.is_contiguous())):
        raise ValueError("the tensors must be contiguous and on one device")
    w = W4Matrix(n, k, k // groups, codes.data_ptr(), scale.data_ptr(),
                 None if zero is None else zero.data_ptr())
    with on_device(dev, stream):
        if workspace is None and T > 16:
            workspace = torch.empty(lib.k3moe_w4_workspace_bytes(ctypes.byref(w), T),
                                    dtype=torch.uint8, device=dev)
        status = call(ctypes.byref(w), T, _DT[x.dtype], _DT[out.dtype], x.data_ptr(), out.data_ptr(),
                      None if workspace is None else workspace.data_ptr(),
                      0 if workspace is None else workspace.numel(), current_stream(dev))
    if status:
        raise K3moeError(status, lib.k3moe_last_error().decode())
    return out


def w4_linear(x, codes, scale, zero=None, out_dtype=None, out=None, workspace=None, stream=None):
    """out [T][n] = x W^T with W[r][j] = (q[r][j] - zero[r][j / g]) * scale[r][j / g]:
    x [T][k] (bf16 or fp32), codes [n][k / 2] uint8 (low nibble = even element),
    scale [n][k / g] bf16, zero [n][k / g] uint8 (None: 8 everywhere).
    out_dtype: bf16 or fp32, x's by default.  workspace: a uint8 tensor of
    k3moe_w4_workspace_bytes (made when needed, above 16 tokens, if not given)."""
    return _run(lib.k3moe_w4_linear, False, x, codes, scale, zero, out_dtype, out, workspace, stream)


def w4_glu(x, codes, scale, zero=None, out_dtype=None, out=None, workspace=None, stream=None):
    """The gated block's first half, silu(x Wg^T) * (x Wu^T) [T][n / 2]: the first
    n / 2 rows of W are the gate, the others the up projection."""
    return _run(lib.k3moe_w4_glu, True, x, codes, scale, zero, out_dtype, out, workspace, stream)
