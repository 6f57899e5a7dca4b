"""Workspace sizes of the routing calls, on the CPU: what is enough for a batch is enough
for a smaller one."""
import pytest

k3 = pytest.importorskip("mxfp4_routed_expert_gemv_amd")

# where a call changes its kernels, and on both sides of it
TOKENS = sorted({t + i for t in (1, 16, 64, 256, 300, 512, 1024, 4096, 1 << 14, (1 << 17) - 64, 1 << 17,
                                 (1 << 17) + 256, 200000, 1 << 19, 1 << 20) for i in (-1, 0, 1) if t + i > 0})


@pytest.mark.parametrize("op", ["OP_PERMUTE", "OP_DISPATCH", "OP_ROUTE_BACKWARD", "OP_LAYER"])
@pytest.mark.parametrize("d,E,k", [(32, 1, 1), (32, 896, 1), (256, 77, 2), (7168, 896, 16), (64, 896, 17),
                                   (32, 1024, 64)])
def test_a_larger_batch_needs_no_less(op, d, E, k):
    sizes = [k3.k3moe_workspace_bytes(k3.make_shape(T, d, 32, E, k, 0, 0, k3.BF16, k3.BF16), getattr(k3, op))
             for T in TOKENS]
    assert sizes == sorted(sizes), [(t, n) for t, n, m in zip(TOKENS, sizes, sizes[1:]) if m < n]
    assert sizes[-1] > 0
