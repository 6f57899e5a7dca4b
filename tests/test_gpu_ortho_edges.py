"""The orthogonalised update of gradients that lie as a program has them, and of more steps
than the usual five."""
import pytest
import torch

from test_gpu_ortho import call, gradient
from test_gpu_routing_edges import inside

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,m,n", [(1, 48, 80), (2, 200, 100), (1, 7, 3), (1, 300, 500)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_and_results_that_begin_inside_another_tensor(batch, m, n, dtype):
    """Matrices of one flat bucket: the same bits as at its beginning, and nothing written
    beside them."""
    g = gradient(batch, m, n, dtype, 40)
    want = call(g)
    at = inside(g)
    assert at.data_ptr() % 16
    assert torch.equal(call(at), want) and torch.equal(at, g)
    bucket = torch.full((g.numel() + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = bucket[1:1 + g.numel()].view(g.shape)
    for src in (g, at):
        out.zero_()
        v = out._version
        assert call(src, out=out) is out and torch.equal(out, want) and out._version > v
        assert float(bucket[0]) == 7.0 and (bucket[1 + g.numel():] == 7.0).all()
    if dtype == torch.bfloat16:   # in place
        assert call(at, out=at) is at and torch.equal(at, want)
        leaf = inside(g).requires_grad_()
        with torch.no_grad():
            assert torch.equal(call(leaf, out=leaf), want) and leaf.requires_grad


def test_overlaps_are_refused_wherever_they_begin():
    from mxfp4_routed_expert_gemv_amd import K3moeError
    buf = torch.zeros(64 * 128 + 64, dtype=torch.bfloat16, device="cuda")
    n = 64 * 128
    for a, b in ((0, 8), (8, 0), (1, 9), (1, 2), (0, 1), (3, 0)):
        g, out = buf[a:a + n].view(64, 128), buf[b:b + n].view(64, 128)
        with pytest.raises((K3moeError, ValueError)):
            call(g, out=out)
    assert not buf.any()


def test_gradients_are_copied_on_the_calls_stream():
    g = gradient(1, 300, 500, torch.bfloat16, 41)
    want = call(g)
    at, out = inside(g), inside(torch.zeros_like(g))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, got2 = call(at, stream=st), call(at, out=out, stream=st)
    st.synchronize()
    assert torch.equal(got, want) and torch.equal(got2, want)
