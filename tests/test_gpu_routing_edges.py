"""Calls of the training through the routing that its documentation allows at the edge
of what it says: operands left out through the C interface, sizes and places in memory
that a user's program comes to."""
import pytest
import torch

from test_gpu_routing import make, randn, routing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,E,k", [(37, 96, 5, 5), (9, 1280, 7, 3), (9, 1312, 7, 3), (300, 2048, 24, 6)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_gradient_of_collect_without_the_other_ones_operands(T, d, E, k, dtype):
    """dw alone reads neither weights nor offsets, drows alone not the rows: NULL then.
    Rows of up to 1280 columns and longer ones have kernels of their own."""
    r = routing()
    from mxfp4_routed_expert_gemv_amd import BF16, F32, k3moe_collect_backward, make_shape
    g, idx, w = make(T, d, E, k, 50, bad=True)
    order = r.sort_pairs(idx, E)
    rows, dy = randn(g, T * k, d, dtype=dtype), randn(g, T, d, dtype=torch.bfloat16)
    drows, dw = r.collect_backward(dy, rows, order, w)
    s = make_shape(T, d, 32, E, k, 0, 0, F32 if dtype == torch.float32 else BF16, BF16)
    only = torch.full_like(dw, 7.0)
    k3moe_collect_backward(s, dy, rows, order.pair_pos, None, None, None, only)
    assert torch.equal(only, dw)
    only = torch.full_like(drows, 7.0)
    k3moe_collect_backward(s, dy, None, order.pair_pos, w, order.offsets, only, None)
    assert torch.equal(only, drows)


@pytest.mark.parametrize("T", [65, 300, 5000])
def test_offsets_that_do_not_ascend_give_no_sums(T):
    """As many chunks as the workspace has room for come only from offsets that ascend."""
    r = routing()
    E, k, d = 12, 4, 96
    g, idx, w = make(T, d, E, k, 51)
    x, wr = randn(g, T, d), randn(g, E, d, dtype=torch.bfloat16)
    dw = randn(g, T, k)
    order = r.sort_pairs(idx, E)
    dx, dwr = r.route_backward(x, wr, idx, w, dw, order)
    assert dwr.any(1).all()
    P = T * k
    for offsets in (order.offsets.flip(0), torch.tensor([0, P] * 6 + [0], dtype=torch.int32, device="cuda")):
        dx2, none = r.route_backward(x, wr, idx, w, dw, order._replace(offsets=offsets.contiguous()))
        assert torch.equal(dx2, dx) and not none.any()


def inside(t):
    """t's values from the second element of a buffer on, in one piece."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    at = buf[1:].view(t.shape)
    at.copy_(t)
    return at


@pytest.mark.parametrize("T", [30, 300])
def test_operands_that_begin_inside_another_tensor(T):
    """Each operand of each call, alone and all of them, at one element of a buffer: the
    same bits as at its beginning."""
    r = routing()
    E, k, d = 9, 3, 96
    g, idx, w = make(T, d, E, k, 52)
    x, wr = randn(g, T, d, dtype=torch.bfloat16), randn(g, E, d, dtype=torch.bfloat16)
    dw, dy, logits = randn(g, T, k), randn(g, T, d, dtype=torch.bfloat16), randn(g, T, E)
    rows, order = r.dispatch(x, idx, E)

    def flat(out):
        if isinstance(out, torch.Tensor):
            return [out]
        return [v for o in out for v in flat(o)]

    def check(call, *operands):
        want = flat(call(*operands))
        for i in range(len(operands) + 1):
            moved = [inside(t) if i in (j, len(operands)) else t for j, t in enumerate(operands)]
            assert all(t.data_ptr() % 16 for t, o in zip(moved, operands) if t is not o)
            assert all(torch.equal(a, b) for a, b in zip(flat(call(*moved)), want)), (call, i)

    check(lambda x, idx: r.dispatch(x, idx, E), x, idx)
    check(lambda idx: r.sort_pairs(idx, E), idx)
    check(lambda rows, pos: r.dispatch_backward(rows, order._replace(pair_pos=pos)), rows, order.pair_pos)
    check(lambda rows, pos, w, add: r.collect(rows, order._replace(pair_pos=pos), w, add=add),
          rows, order.pair_pos, w, x)
    check(lambda dy, rows, pos, w, off: r.collect_backward(dy, rows, order._replace(pair_pos=pos, offsets=off), w),
          dy, rows, order.pair_pos, w, order.offsets)
    check(lambda x, wr, idx, w, dw, lg, off, pairs, pos: r.route_backward(
        x, wr, idx, w, dw, r.Order(order.counts, off, pairs, pos), "sigmoid_norm", lg),
          x, wr, idx, w, dw, logits, order.offsets, order.sorted_pair, order.pair_pos)


def test_micro_batches_of_one_choice():
    """Tokens 5 .. of a routed batch: their weights begin at 5 * 3 * 4 = 60 bytes."""
    r = routing()
    T, d, E, k, at = 40, 96, 7, 3, 5
    g, *_ = make(T, d, E, k, 53)
    x = randn(g, T, d, dtype=torch.bfloat16).requires_grad_()
    bias = inside(randn(g, E, std=0.1))
    wr = inside(randn(g, E, d, dtype=torch.bfloat16, std=0.1)).requires_grad_()
    idx, w = r.route_tokens(inside(x.detach()).requires_grad_(), wr, k, "sigmoid_norm", bias)
    i2, w2 = r.route_tokens(x, wr.detach().clone().requires_grad_(), k, "sigmoid_norm", bias.clone())
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    up = randn(g, T - at, d, dtype=torch.bfloat16)

    def step(x, idx, w):
        rows, order = r.dispatch_tokens(x, idx, E)
        y = r.collect_tokens(rows, order, w, add=x)
        return (y, *torch.autograd.grad(y, (x, w), up))
    part = [t.detach()[at:] for t in (x, w)]
    assert part[1].data_ptr() % 16
    got = step(part[0].requires_grad_(), idx[at:], part[1].requires_grad_())
    want = step(part[0].detach().clone().requires_grad_(), idx[at:].clone(), part[1].detach().clone().requires_grad_())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_operands_are_copied_on_the_calls_stream():
    r = routing()
    T, d, E, k = 300, 512, 24, 6
    g, idx, w = make(T, d, E, k, 54)
    x, off = randn(g, T, d, dtype=torch.bfloat16), inside(idx)
    want, order = r.dispatch(x, idx, E)
    y = r.collect(want, order, w)
    st = torch.cuda.Stream()
    w = inside(w)
    st.wait_stream(torch.cuda.current_stream())
    rows, o2 = r.dispatch(x, off, E, stream=st)
    got = r.collect(rows, o2, w, stream=st)
    st.synchronize()
    assert torch.equal(rows, want) and torch.equal(got, y)


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_collect_as_an_operation_into_another_type(dtype, out):
    """The bits of collect and of its backward with y and dy in the given type."""
    r = routing()
    T, d, E, k = 70, 96, 9, 3
    g, idx, w = make(T, d, E, k, 55)
    order = r.sort_pairs(idx, E)
    rows, w = randn(g, T * k, d, dtype=dtype).requires_grad_(), w.requires_grad_()
    y = r.collect_tokens(rows, order, w, out_dtype=out)
    assert y.dtype == out and torch.equal(y, r.collect(rows.detach(), order, w.detach(), out_dtype=out))
    up = randn(g, T, d, dtype=out)
    got = torch.autograd.grad(y, (rows, w), up)
    want = r.collect_backward(up, rows.detach(), order, w.detach())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    add = randn(g, T, d, dtype=out).requires_grad_()
    y = r.collect_tokens(rows, order, w, add, out)
    assert torch.equal(torch.autograd.grad(y, add, up)[0], up)


@pytest.mark.parametrize("T", [5, 300])
def test_the_c_interfaces_own_wrappers(T):
    """The package's k3moe_* functions of these calls, on the caller's buffers: what the
    calls above return."""
    r = routing()
    import mxfp4_routed_expert_gemv_amd as k3
    d, E, k = 96, 9, 3
    g, idx, w = make(T, d, E, k, 56, bad=True)
    x, wr = randn(g, T, d, dtype=torch.bfloat16), randn(g, E, d, dtype=torch.bfloat16)
    dw, dy = randn(g, T, k), randn(g, T, d, dtype=torch.bfloat16)
    s = k3.make_shape(T, d, 32, E, k, 0, 0, k3.BF16, k3.BF16)

    def scratch(op):
        return torch.empty(k3.k3moe_workspace_bytes(s, op), dtype=torch.uint8, device="cuda")

    def new(*shape, dtype=torch.bfloat16):
        return torch.full(shape, 7, dtype=dtype, device="cuda")
    want, order = r.dispatch(x, idx, E)
    rows, parts = new(T * k, d), [new(*o.shape, dtype=torch.int32) for o in order]
    k3.k3moe_dispatch(s, x, idx, rows, *parts, None, scratch(k3.OP_DISPATCH))
    assert torch.equal(rows, want) and all(torch.equal(a, b) for a, b in zip(parts, order))
    dx = new(T, d)
    k3.k3moe_dispatch_backward(s, rows, order.pair_pos, dx)
    assert torch.equal(dx, r.dispatch_backward(rows, order))
    y = new(T, d)
    k3.k3moe_collect(s, rows, order.pair_pos, w, x, y)
    assert torch.equal(y, r.collect(rows, order, w, add=x))
    drows, dwc = new(T * k, d), new(T, k, dtype=torch.float32)
    k3.k3moe_collect_backward(s, dy, rows, order.pair_pos, w, order.offsets, drows, dwc)
    assert all(torch.equal(a, b) for a, b in zip((drows, dwc), r.collect_backward(dy, rows, order, w)))
    dwr = new(E, d)
    k3.k3moe_route_backward(s, x, wr, idx, w, dw, None, order.offsets, order.sorted_pair, order.pair_pos, dx, dwr,
                            scratch(k3.OP_ROUTE_BACKWARD))
    assert all(torch.equal(a, b) for a, b in zip((dx, dwr), r.route_backward(x, wr, idx, w, dw, order)))
