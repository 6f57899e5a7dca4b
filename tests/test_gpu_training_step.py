"""Steps of training a small layer, all of it through the library but the routed
experts' own products: route, dispatch, collect beside the shared experts, their
backward, the norm and clipping of the gradients, the orthogonalised update.

Tolerances.  The loss is sum(y c) with c exact in bf16, so dL/dy = c: nothing of the
backward goes through y's rounding.  Each gradient's error in norm stays under
2^-8 sqrt(r) of it for the r roundings to bf16 on its way (as the shared experts'
own tests have it; the products beside are fp32)."""
import math

import pytest
import torch

from gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu

F8 = torch.float64
T, D, FS, S, E, K = 200, 128, 64, 2, 12, 3


class Layer:
    def __init__(self, seed, router):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std=1.0, dtype=torch.bfloat16):
            return (torch.randn(shape, generator=g) * std).to(dtype).cuda().requires_grad_()
        self.router = router
        self.w_router = normal(E, D, std=0.2)
        self.w13, self.w2 = normal(S, 2 * FS, D, std=0.09), normal(S, D, FS, std=0.12)
        self.experts = normal(E, D, D, std=0.09, dtype=torch.float32)
        self.x = normal(T, D)
        self.c = normal(T, D).detach()
        self.weights = [self.w_router, self.w13, self.w2, self.experts]

    def routed(self, rows, order):
        # (every row through every expert, one of the results taken: no sizes on the host)
        of = torch.searchsorted(order.offsets[1:].contiguous(),
                                torch.arange(T * K, dtype=torch.int32, device="cuda"), right=True)
        every = torch.matmul(rows.float()[None], self.experts)   # [E][T k][D]
        return every.gather(0, of.long().clamp(max=E - 1)[None, :, None].expand(1, T * K, D))[0]

    def forward(self):
        from mxfp4_routed_expert_gemv_amd.routing import collect_tokens, dispatch_tokens, route_tokens
        from mxfp4_routed_expert_gemv_amd.shared import shared_ffn
        idx, w = route_tokens(self.x, self.w_router, K, self.router)
        rows, order = dispatch_tokens(self.x, idx, E)
        return collect_tokens(self.routed(rows, order), order, w, add=shared_ffn(self.x, self.w13, self.w2)), idx

    def reference(self, idx):
        x, wr, w13, w2, ex = (t.detach().to(F8).requires_grad_() for t in (self.x, *self.weights))
        logits = (x @ wr.t()).gather(1, idx.long())
        w = torch.softmax(logits, 1) if self.router == "softmax" else torch.sigmoid(logits)
        if self.router == "sigmoid_norm":
            w = w / w.sum(1, keepdim=True)
        y = 0
        for j in range(S):
            g, u = (x @ w13[j].t()).chunk(2, 1)
            y = y + (g * torch.sigmoid(g) * u) @ w2[j].t()
        for s in range(K):
            y = y + w[:, s, None] * (x[:, None] @ ex[idx[:, s].long()])[:, 0]
        (y * self.c.to(F8)).sum().backward()
        return y.detach(), x.grad, [t.grad for t in (wr, w13, w2, ex)]


def layer(seed, router="softmax"):
    require_gpu()
    return Layer(seed, router)


def near(got, want, roundings, name):
    rel = float((got.to(F8) - want).norm() / want.norm())
    log(f"  {name}: {rel:.1e}, allowed {2.0 ** -8 * math.sqrt(roundings):.1e}")
    assert rel <= 2.0 ** -8 * math.sqrt(roundings), name


@pytest.mark.parametrize("router", ["softmax", "sigmoid", "sigmoid_norm"])
def test_gradients_of_a_step(router):
    L = layer(1, router)
    y, idx = L.forward()
    (y.float() * L.c.float()).sum().backward()
    want_y, want_x, want = L.reference(idx)
    near(y.detach(), want_y, 4, "y")                # gu, h, the shared experts' y, y
    near(L.x.grad, want_x, 9, "dx")                 # gu, h, dg, du, three parts and two sums
    for t, w, r, name in zip(L.weights, want, (1, 5, 5, 1), ("dw_router", "dw13", "dw2", "dexperts")):
        near(t.grad, w, r, name)


def test_steps_with_clipping_and_orthogonalised_updates():
    """Three steps; every update is the formula's on the gradients at hand: the clipped
    ones through the steps in 64 bits, for stacks and for the flat router."""
    from mxfp4_routed_expert_gemv_amd.grads import clip_grads
    from mxfp4_routed_expert_gemv_amd.ortho import orthogonalize
    import test_gpu_ortho as o
    L = layer(2)
    trained = [L.w_router, L.w13, L.w2]
    for step in range(3):
        for t in [L.x, *L.weights]:
            t.grad = None
        y, _ = L.forward()
        (y.float() * L.c.float()).sum().backward()
        grads = [t.grad for t in trained]
        before = [g.to(F8) for g in grads]
        norm = clip_grads(grads, 1.0)
        total = math.sqrt(sum(float(g.square().sum()) for g in before))
        assert abs(float(norm) / total - 1) < 1e-5
        factor = min(1.0, 1.0 / total)
        for g, b in zip(grads, before):
            near(g, b * factor, 1, "clipped")
        for t, g in zip(trained, grads):
            update = orthogonalize(g)
            stack = g if g.dim() == 3 else g[None]
            want, model = o.exact(stack), o.rounded(stack)
            cost = float((model.to(torch.bfloat16).to(F8) - want).norm())
            assert float((update.view_as(stack).to(F8) - want).norm()) <= 1.25 * cost
            old = t.detach().clone()
            with torch.no_grad():
                t.add_(update, alpha=-0.02)
            assert not torch.equal(t, old) and torch.isfinite(t).all()


def test_a_step_captured_and_replayed():
    """Forward, backward, clipping and updates of one step in a graph; replays on new
    tokens against the same step without one."""
    from mxfp4_routed_expert_gemv_amd.grads import clip_grads
    from mxfp4_routed_expert_gemv_amd.ortho import orthogonalize

    def step(L):
        y, _ = L.forward()
        grads = torch.autograd.grad((y.float() * L.c.float()).sum(), [L.w_router, L.w13, L.w2])
        grads = [g.clone() for g in grads]
        norm = clip_grads(grads, 1.0)
        return y.detach(), norm, *(orthogonalize(g) for g in grads)
    L = layer(3)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(L)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(L)
    for i in range(4):
        M = layer(10 + i)
        with torch.no_grad():
            L.x.copy_(M.x)
            L.c.copy_(M.c)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for a, b, name in zip(got, step(L), ("y", "norm", "router", "w13", "w2")):
            assert torch.equal(a, b), (i, name)
