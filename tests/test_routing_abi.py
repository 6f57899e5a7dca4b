"""Argument checks of the calls that train through the routing, on the CPU: every
invalid call is refused with the documented status before anything is launched."""
import ctypes

import pytest
import torch

k3 = pytest.importorskip("mxfp4_routed_expert_gemv_amd")

EINVAL, ESHAPE, EALIGN, EWORKSPACE, EUNSUPPORTED = 1, 2, 3, 4, 5
# aligned addresses that are never dereferenced (validation fails first), far apart
A = {n: 0x10000000 * (i + 1) for i, n in enumerate(
    ("x", "idx", "rows", "counts", "offsets", "sorted_pair", "pair_pos", "ws", "dy", "w", "dw",
     "drows", "dx", "y", "add", "wr", "dwr", "logits", "diag"))}
BIG = 1 << 24


def shape(T=8, **kw):
    a = dict(T=T, d=256, f=32, E=16, k=4, n_shared=0, f_shared=0, x_dtype=k3.BF16, out_dtype=k3.BF16)
    a.update(kw)
    return k3.make_shape(**a)


NAMES = {
    "dispatch": ("x", "idx", "rows", "counts", "offsets", "sorted_pair", "pair_pos", "diag", "ws"),
    "dispatch_backward": ("drows", "pair_pos", "dx"),
    "collect": ("rows", "pair_pos", "w", "add", "y"),
    "collect_backward": ("dy", "rows", "pair_pos", "w", "offsets", "drows", "dw"),
    "route_backward": ("x", "wr", "idx", "w", "dw", "logits", "offsets", "sorted_pair", "pair_pos",
                       "dx", "dwr", "ws"),
}
WRITTEN = {"dispatch": ("rows", "counts", "offsets", "sorted_pair", "pair_pos", "ws"),
           "dispatch_backward": ("dx",), "collect": ("y",), "collect_backward": ("drows", "dw"),
           "route_backward": ("dx", "dwr", "ws")}
OPTIONAL = {"diag", "add", "logits"}


def call(op, s, ws_bytes=BIG, **kw):
    p = {**A, "diag": None, "logits": A["logits"] if s is not None and s.router == 2 else None, **kw}
    args = []
    for n in NAMES[op]:
        args.append(p[n])
        if n == "ws":
            args.append(ws_bytes)
    return getattr(k3.lib, f"k3moe_{op}")(ctypes.byref(s) if s is not None else None, *args, None)


@pytest.mark.parametrize("op", NAMES)
def test_refusals(op):
    def shape(T=300, **kw):   # (a batch that needs the workspace)
        return globals()["shape"](T=T, **kw)
    assert call(op, None) == EINVAL
    assert call(op, shape(T=-1)) == EINVAL
    assert call(op, shape(d=250)) == ESHAPE
    assert call(op, shape(E=2000)) == ESHAPE
    assert call(op, shape(k=17)) == ESHAPE
    assert call(op, shape(T=1 << 30)) == ESHAPE
    assert call(op, shape(x_dtype=2)) == EUNSUPPORTED
    assert call(op, shape(out_dtype=2)) == EUNSUPPORTED
    may_be_null = OPTIONAL | ({"drows", "dw"} if op == "collect_backward" else set()) | (
        {"dx", "dwr"} if op == "route_backward" else set())
    for n in NAMES[op]:
        if n not in may_be_null:
            assert call(op, shape(), **{n: None}) == (EWORKSPACE if n == "ws" else EINVAL), n
        if n != "logits":
            assert call(op, shape(), **{n: A[n] + 8}) == EALIGN, n
    # nothing that is written may touch another operand
    for n in WRITTEN[op]:
        for m in NAMES[op]:
            if m != n and m not in OPTIONAL:
                assert call(op, shape(), **{n: A[m]}) == EINVAL, (n, m)
    if "ws" in NAMES[op]:
        assert call(op, shape(T=3000), ws_bytes=16) == EWORKSPACE
        assert call(op, shape(T=3000), ws=A["ws"] + 16) == EALIGN


@pytest.mark.parametrize("op", NAMES)
def test_empty_batch(op):
    s = shape(T=0)
    assert call(op, s, ws_bytes=0, **{n: None for n in NAMES[op]}) == 0


def test_outputs_that_are_not_wanted():
    s = shape()
    assert call("collect_backward", s, drows=None, dw=None) == 0
    assert call("collect_backward", s, drows=None, rows=None) == EINVAL
    assert call("collect_backward", s, dw=None, w=None) == EINVAL
    assert call("collect_backward", s, dw=None, offsets=None) == EINVAL
    assert call("route_backward", s, dx=None, dwr=None) == 0


def test_the_renormalised_router_needs_logits():
    assert call("route_backward", shape(router=k3.ROUTER_SIGMOID_NORM), logits=None) == EINVAL
    assert call("route_backward", shape(router=k3.ROUTER_SIGMOID_NORM), logits=A["logits"] + 4) == EALIGN
    assert call("route_backward", shape(), logits=A["logits"]) == EINVAL
    assert call("route_backward", shape(router=k3.ROUTER_SIGMOID), logits=A["logits"]) == EINVAL


def test_workspace():
    assert k3.k3moe_workspace_bytes(shape(), k3.OP_DISPATCH) == 0   # (one launch)
    for T, k in ((257, 4), (256, 16)):
        s = shape(T=T, k=k)
        need = 0 if T == 256 else k3.k3moe_workspace_bytes(s, k3.OP_PERMUTE)
        assert k3.k3moe_workspace_bytes(s, k3.OP_DISPATCH) == need
    assert k3.k3moe_workspace_bytes(shape(T=64), k3.OP_ROUTE_BACKWARD) == 0
    s = shape(T=3000)
    assert k3.k3moe_workspace_bytes(s, k3.OP_ROUTE_BACKWARD) >= 4 * 3000 * 4 + 2 * 46 * 256 * 4
    assert k3.k3moe_workspace_bytes(shape(T=0), k3.OP_ROUTE_BACKWARD) == 0
    assert k3.k3moe_workspace_bytes(shape(d=100), k3.OP_ROUTE_BACKWARD) == 0


def test_python_calls_refuse_what_is_not_on_a_gpu():
    from mxfp4_routed_expert_gemv_amd import routing as r
    x, idx, w = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    order = r.Order(torch.zeros(8, dtype=torch.int32), torch.zeros(9, dtype=torch.int32),
                    torch.zeros(8, dtype=torch.int32), idx)
    rows, wr = torch.zeros(8, 64), torch.zeros(8, 64, dtype=torch.bfloat16)
    for f in (lambda: r.dispatch(x, idx, 8), lambda: r.sort_pairs(idx, 8),
              lambda: r.dispatch_backward(rows, order), lambda: r.collect(rows, order, w),
              lambda: r.collect_backward(x, rows, order, w),
              lambda: r.route_backward(x, wr, idx, w, w, order),
              lambda: r.route_tokens(x, wr, 2), lambda: r.dispatch(x[0], idx, 8),
              lambda: r.collect(rows[0], order, w), lambda: r.sort_pairs(idx[0], 8),
              lambda: r.route_tokens(x, wr, 2, router="none")):
        with pytest.raises(ValueError):
            f()
