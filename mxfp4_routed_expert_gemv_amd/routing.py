"""Training through the routing: rows of tokens sorted by expert and back, with
the weights applied, and the gradients of both and of the router; each as plain
calls and as torch operations that autograd goes through.

Tensors are torch device tensors, contiguous, all on one device; the work is
enqueued on that device's current stream (or `stream`).  An operand that begins
inside another tensor, at other than 16 bytes, is copied first.  Every computation
happens in libk3moe's kernels; this file only marshals."""
from collections import namedtuple
from ctypes import byref
from functools import lru_cache

import torch

from . import (BF16, DIAG_COUNT, F32, OP_DISPATCH, OP_PERMUTE, OP_ROUTE, OP_ROUTE_BACKWARD,
               ROUTERS, _addr, _check, _ws, check_workspace, k3moe_permute, k3moe_route,
               k3moe_workspace_bytes, lib, make_shape, on_device)

_DT = {torch.float32: F32, torch.bfloat16: BF16}

# Where the (token, slot) pairs lie by expert, as k3moe_permute says: counts [E], offsets
# [E + 1], sorted_pair [T k] and pair_pos [T][k] (-1: a pair without a row), int32.
Order = namedtuple("Order", "counts offsets sorted_pair pair_pos")


@lru_cache(maxsize=256)
def _shape_of(T, d, E, k, x_dtype, out_dtype, router=0, op=None):
    # the experts' own sizes are not used by these calls
    shape = make_shape(T, d, 32, E, k, 0, 0, _DT[x_dtype], _DT[out_dtype], router)
    return shape, 0 if op is None else k3moe_workspace_bytes(shape, op)


_raw_stream = torch._C._cuda_getCurrentRawStream
_ptr = torch.Tensor.data_ptr


def _need(t, name, shape, dtypes, device):
    if t.dtype not in dtypes:
        raise TypeError(f"{name} is {t.dtype}; {' or '.join(map(str, dtypes))} is needed")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; {tuple(shape)} is needed")
    index = t.get_device()
    if index < 0 or index != device.index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on the operands' GPU")


def _whole(*operands):
    """The operands at 16 bytes, as the calls need them: a contiguous part of a larger
    tensor (a micro-batch's rows of w, a gradient that autograd hands over) may begin at
    any element.  Called where the call's stream is current, which the copies belong to."""
    for t in operands:
        if t is not None and t.data_ptr() & 15:
            return [t if t is None or not t.data_ptr() & 15 else t.clone() for t in operands]
    return operands


def _sizes(pair_pos, rows, name):
    if pair_pos.dim() != 2 or rows.dim() != 2:
        raise ValueError(f"pair_pos {tuple(pair_pos.shape)} is [T][k] and {name} "
                         f"{tuple(rows.shape)} is [T k][d]")
    return (*pair_pos.shape, rows.shape[1])


def _out(dtype, name):
    if dtype not in _DT:
        raise TypeError(f"{name} is float32 or bfloat16, not {dtype}")
    return dtype


def _scratch(workspace, nbytes, dev):
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    check_workspace(workspace, dev.index)
    return workspace


_I32, _F = (torch.int32,), (torch.float32,)


def _empty_order(T, k, E, dev):
    # one allocation, every part at 16 bytes
    P, e4, p4 = T * k, E + 3 & ~3, T * k + 3 & ~3
    buf = (torch.empty if T else torch.zeros)(2 * e4 + 4 + 2 * p4, dtype=torch.int32, device=dev)
    s = torch.as_strided
    return Order(s(buf, (E,), (1,), 0), s(buf, (E + 1,), (1,), e4), s(buf, (P,), (1,), 2 * e4 + 4),
                 s(buf, (T, k), (k, 1), 2 * e4 + 4 + p4))


def _check_ids(idx, diag, dev):
    _need(idx, "idx", idx.shape, _I32, dev)
    if diag is not None:
        _need(diag, "diag", (DIAG_COUNT,), _I32, dev)


def sort_pairs(idx, n_experts, diag=None, workspace=None, stream=None):
    """The Order of idx [T][k] int32: dispatch without the rows."""
    if idx.dim() != 2:
        raise ValueError(f"idx {tuple(idx.shape)} is [T][k]")
    (T, k), dev, E = idx.shape, idx.device, n_experts
    _check_ids(idx, diag, dev)
    shape, nbytes = _shape_of(T, 32, E, k, torch.bfloat16, torch.bfloat16, op=OP_PERMUTE)
    with on_device(dev, stream):
        idx, = _whole(idx)
        order = _empty_order(T, k, E, dev)
        k3moe_permute(shape, idx, *order, diag, _scratch(workspace, nbytes, dev),
                      _raw_stream(dev.index))
    return order


def dispatch(x, idx, n_experts, diag=None, workspace=None, stream=None):
    """rows [T k][d], x's rows sorted by expert (stable; zeros behind the last), and
    their Order.  x [T][d] bf16 or fp32; idx [T][k] int32, the experts of every token:
    an id outside [0, n_experts), or an earlier slot's, has no row."""
    if x.dim() != 2 or idx.dim() != 2:
        raise ValueError(f"x {tuple(x.shape)} is [T][d] and idx {tuple(idx.shape)} is [T][k]")
    (T, d), k, dev, E = x.shape, idx.shape[1], x.device, n_experts
    _need(x, "x", (T, d), _DT, dev)
    if idx.shape[0] != T:
        raise ValueError(f"x {tuple(x.shape)} and idx {tuple(idx.shape)} differ in tokens")
    _check_ids(idx, diag, dev)
    shape, nbytes = _shape_of(T, d, E, k, x.dtype, x.dtype, op=OP_DISPATCH)
    with on_device(dev, stream):
        x, idx = _whole(x, idx)
        rows = torch.empty((T * k, d), dtype=x.dtype, device=dev)
        order = _empty_order(T, k, E, dev)
        ws = _scratch(workspace, nbytes, dev)
        _check(lib.k3moe_dispatch(byref(shape), _ptr(x), _ptr(idx), _ptr(rows), *map(_ptr, order),
                                  _addr(diag), *_ws(ws), _raw_stream(dev.index)))
    return rows, order


def dispatch_backward(drows, order, out_dtype=None, stream=None):
    """dx [T][d]: each token's rows of drows [T k][d] summed.  out_dtype: drows's by
    default."""
    pair_pos = order[3]
    T, k, d = _sizes(pair_pos, drows, "drows")
    dev, out_dtype = drows.device, _out(out_dtype or drows.dtype, "dx")
    _need(drows, "drows", (T * k, d), _DT, dev)
    _need(pair_pos, "pair_pos", (T, k), _I32, dev)
    shape, _ = _shape_of(T, d, k, k, drows.dtype, out_dtype)
    with on_device(dev, stream):
        drows, pair_pos = _whole(drows, pair_pos)
        dx = torch.empty((T, d), dtype=out_dtype, device=dev)
        _check(lib.k3moe_dispatch_backward(byref(shape), _ptr(drows), _ptr(pair_pos), _ptr(dx),
                                           _raw_stream(dev.index)))
    return dx


def collect(rows, order, w, add=None, out_dtype=None, stream=None):
    """y [T][d] = add + the sum over each token's slots of w * its row: rows [T k][d]
    (bf16 or fp32) as dispatch sorted them, w [T][k] fp32, add [T][d] in y's type or
    None.  Slots of weight 0 are skipped.  out_dtype: add's by default, or rows's."""
    pair_pos = order[3]
    T, k, d = _sizes(pair_pos, rows, "rows")
    dev = rows.device
    out_dtype = _out(out_dtype or (rows if add is None else add).dtype, "y")
    _need(rows, "rows", (T * k, d), _DT, dev)
    _need(pair_pos, "pair_pos", (T, k), _I32, dev)
    _need(w, "w", (T, k), _F, dev)
    if add is not None:
        _need(add, "add", (T, d), (out_dtype,), dev)
    shape, _ = _shape_of(T, d, k, k, rows.dtype, out_dtype)
    with on_device(dev, stream):
        rows, pair_pos, w, add = _whole(rows, pair_pos, w, add)
        y = torch.empty((T, d), dtype=out_dtype, device=dev)
        _check(lib.k3moe_collect(byref(shape), _ptr(rows), _ptr(pair_pos), _ptr(w), _addr(add),
                                 _ptr(y), _raw_stream(dev.index)))
    return y


def collect_backward(dy, rows, order, w, need=(True, True), stream=None):
    """drows [T k][d] (rows's type) and dw [T][k] fp32 from dy [T][d]; None in the
    place of one that `need` leaves out."""
    _, offsets, _, pair_pos = order
    T, k, d = _sizes(pair_pos, rows, "rows")
    dev = rows.device
    E = offsets.numel() - 1
    _need(rows, "rows", (T * k, d), _DT, dev)
    _need(dy, "dy", (T, d), _DT, dev)
    _need(pair_pos, "pair_pos", (T, k), _I32, dev)
    _need(offsets, "offsets", (E + 1,), _I32, dev)
    _need(w, "w", (T, k), _F, dev)
    shape, _ = _shape_of(T, d, E, k, rows.dtype, dy.dtype)
    with on_device(dev, stream):
        dy, rows, pair_pos, w, offsets = _whole(dy, rows, pair_pos, w, offsets)
        drows = torch.empty_like(rows) if need[0] else None
        dw = torch.empty((T, k), dtype=torch.float32, device=dev) if need[1] else None
        _check(lib.k3moe_collect_backward(byref(shape), _ptr(dy), _ptr(rows), _ptr(pair_pos),
                                          _ptr(w), _ptr(offsets), _addr(drows), _addr(dw),
                                          _raw_stream(dev.index)))
    return drows, dw


def route_backward(x, w_router, idx, w, dw, order, router="softmax", logits=None,
                   dw_dtype=torch.bfloat16, need=(True, True), workspace=None, stream=None):
    """dx [T][d] (x's type) and dw_router [E][d] (dw_dtype) from dw [T][k], the
    gradient of the weights w [T][k] that the router gave the experts idx [T][k];
    None in the place of one that `need` leaves out.  order: the Order of idx.
    logits [T][E] fp32: for "sigmoid_norm"."""
    _, offsets, sorted_pair, pair_pos = order
    if x.dim() != 2 or w_router.dim() != 2 or idx.dim() != 2:
        raise ValueError(f"x {tuple(x.shape)} is [T][d], w_router {tuple(w_router.shape)} is [E][d] "
                         f"and idx {tuple(idx.shape)} is [T][k]")
    if router not in ROUTERS:
        raise ValueError(f"router is one of {', '.join(ROUTERS)}, not {router!r}")
    (T, d), E, k, dev = x.shape, w_router.shape[0], idx.shape[1], x.device
    _need(x, "x", (T, d), _DT, dev)
    _need(w_router, "w_router", (E, d), (torch.bfloat16,), dev)
    for t, name, size, types in ((idx, "idx", (T, k), _I32), (w, "w", (T, k), _F),
                                 (dw, "dw", (T, k), _F), (offsets, "offsets", (E + 1,), _I32),
                                 (sorted_pair, "sorted_pair", (T * k,), _I32),
                                 (pair_pos, "pair_pos", (T, k), _I32)):
        _need(t, name, size, types, dev)
    if logits is not None:
        _need(logits, "logits", (T, E), _F, dev)
    shape, nbytes = _shape_of(T, d, E, k, x.dtype, _out(dw_dtype, "dw_router"), ROUTERS[router],
                              OP_ROUTE_BACKWARD)
    with on_device(dev, stream):
        x, w_router, idx, w, dw, logits, offsets, sorted_pair, pair_pos = _whole(
            x, w_router, idx, w, dw, logits, offsets, sorted_pair, pair_pos)
        dx = torch.empty_like(x) if need[0] else None
        dwr = torch.empty((E, d), dtype=dw_dtype, device=dev) if need[1] else None
        # (an empty tensor's address may be NULL: for T = 0 nothing is read or written there)
        ws = _scratch(workspace, nbytes, dev)
        _check(lib.k3moe_route_backward(byref(shape), _ptr(x), _ptr(w_router), _ptr(idx), _ptr(w),
                                        _ptr(dw), _addr(logits), _ptr(offsets), _ptr(sorted_pair),
                                        _ptr(pair_pos), _addr(dx) if T else None, _addr(dwr),
                                        *_ws(ws), _raw_stream(dev.index)))
    return dx, dwr


# ------------------------------------------------------------- torch operations
class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, idx, n_experts):
        rows, order = dispatch(x, idx, n_experts)
        ctx.save_for_backward(*order)
        ctx.mark_non_differentiable(*order)
        return (rows, *order)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, drows, *_):
        return dispatch_backward(drows.contiguous(), ctx.saved_tensors), None, None


class _Collect(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, w, add, out_dtype, *order):
        ctx.save_for_backward(rows, w, *order)
        return collect(rows, order, w, add, out_dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        rows, w, *order = ctx.saved_tensors
        dy = dy.contiguous()
        drows, dw = collect_backward(dy, rows, order, w, need=ctx.needs_input_grad[:2])
        return (drows, dw, dy if ctx.needs_input_grad[2] else None, None, None, None, None, None)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_router, k, router, bias, diag):
        (T, d), E, dev = x.shape, w_router.shape[0], x.device
        shape, nbytes = _shape_of(T, d, E, k, x.dtype, w_router.dtype, ROUTERS[router], OP_ROUTE)
        with on_device(dev):
            idx = torch.empty((T, k), dtype=torch.int32, device=dev)
            w = torch.empty((T, k), dtype=torch.float32, device=dev)
            logits = (torch.empty((T, E), dtype=torch.float32, device=dev)
                      if router == "sigmoid_norm" else None)
            at, wr, bias = _whole(x, w_router, bias)
            k3moe_route(shape, at, wr, idx, w, logits, diag, _scratch(None, nbytes, dev),
                        _raw_stream(dev.index), router_bias=bias)
        ctx.save_for_backward(x, w_router, idx, w, logits)
        ctx.router = router
        ctx.mark_non_differentiable(idx)
        return idx, w

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _, dw):
        x, w_router, idx, w, logits = ctx.saved_tensors
        # the order of the pairs, sorted again from the ids rather than kept
        order = sort_pairs(idx, w_router.shape[0])
        dx, dwr = route_backward(x, w_router, idx, w, dw.contiguous(), order, ctx.router, logits,
                                 need=ctx.needs_input_grad[:2])
        return dx, dwr, None, None, None, None


def route_tokens(x, w_router, k, router="softmax", router_bias=None, diag=None):
    """k3moe_route as a torch operation: idx [T][k] int32 and w [T][k] fp32,
    differentiable once in x and w_router [E][d] bf16 through w (the choice of the
    experts has no gradient, and neither has router_bias, which only bends it)."""
    if router not in ROUTERS:
        raise ValueError(f"router is one of {', '.join(ROUTERS)}, not {router!r}")
    if x.dim() != 2 or w_router.dim() != 2:
        raise ValueError(f"x {tuple(x.shape)} is [T][d] and w_router {tuple(w_router.shape)} is [E][d]")
    _need(x, "x", x.shape, _DT, w_router.device)
    _need(w_router, "w_router", (w_router.shape[0], x.shape[1]), (torch.bfloat16,), x.device)
    if router_bias is not None:
        _need(router_bias, "router_bias", (w_router.shape[0],), _F, x.device)
    if diag is not None:
        _need(diag, "diag", (DIAG_COUNT,), _I32, x.device)
    return _Route.apply(x, w_router, k, router, router_bias, diag)


def dispatch_tokens(x, idx, n_experts):
    """dispatch as a torch operation: rows, differentiable once in x, and their Order."""
    rows, *order = _Dispatch.apply(x, idx, n_experts)
    return rows, Order(*order)


def collect_tokens(rows, order, w, add=None, out_dtype=None):
    """collect as a torch operation: y, differentiable once in rows, w and add."""
    return _Collect.apply(rows, w, add, out_dtype, *order)
