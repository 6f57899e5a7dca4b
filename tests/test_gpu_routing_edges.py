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
