"""Rows to the experts' order and back, their gradients and the router's, on the
GPU against their definitions in 64 bits.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value, an fp32 sum
of n terms by at most n 2^-24 of the sum of the terms' magnitudes; a bound adds
the errors of what it is made from, each weighted with what it is multiplied
with.  Moved rows and positions are equal, bit for bit."""
import pytest
import torch

from gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu

B, S24 = 2.0 ** -8, 2.0 ** -24
F8 = torch.float64
DTS = [torch.bfloat16, torch.float32]
# T, d, E, k: one token and one expert; toy; odd counts; more than the small sort takes;
# one expert for many tokens; many slots; the full-size row
SIZES = [(1, 32, 1, 1), (4, 256, 16, 4), (37, 96, 5, 5), (257, 544, 19, 3), (700, 64, 3, 1),
         (65, 160, 130, 64), (64, 160, 130, 64), (23, 7168, 896, 16), (1100, 1056, 40, 10), (5, 16384, 7, 2)]


def routing():
    require_gpu()
    from mxfp4_routed_expert_gemv_amd import routing as r
    return r


def make(T, d, E, k, seed, bad=False, skew=False):
    """ids in ascending order, some outside the range or repeated (bad), weights."""
    g = torch.Generator().manual_seed(seed)
    score = torch.rand((T, E), generator=g)
    if skew:
        score[:, 0] += 1.0
    idx = score.topk(k).indices.sort(1).values.int()
    if bad:
        idx[::3, -1] = -1
        idx[1::4, 0] = E
        if k > 1:
            idx[2::5, 1] = idx[2::5, 0]
        idx[T - T // 4:] = -1
    w = torch.softmax(torch.randn((T, k), generator=g), 1)
    return g, idx.cuda(), w.cuda()


def randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def positions(idx, E):
    """counts, offsets, sorted_pair, pair_pos by a loop over the pairs."""
    rows = idx.tolist()
    by = [[] for _ in range(E)]
    for t, row in enumerate(rows):
        for s, e in enumerate(row):
            if 0 <= e < E and e not in row[:s]:
                by[e].append(t * len(row) + s)
    order = [p for b in by for p in b]
    P = idx.numel()
    pos = [-1] * P
    for q, p in enumerate(order):
        pos[p] = q
    counts = [len(b) for b in by]
    offsets = [sum(counts[:e]) for e in range(E + 1)]
    return (torch.tensor(counts), torch.tensor(offsets), torch.tensor(order + [-1] * (P - len(order))),
            torch.tensor(pos).view(idx.shape))


def within(got, want, tol, name):
    assert got.shape == want.shape, (name, got.shape, want.shape)
    err = (got.to(F8) - want).abs()
    worst = float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0
    log(f"  {name}: worst error {worst:.3f} of its bound")
    assert worst <= 1.0, f"{name}: {worst:.3f} times its bound"


def step(t, dtype):
    return (B if dtype == torch.bfloat16 else S24) * t.abs()


def gathered(rows, pos):
    """[T][k][d] in 64 bits, zeros for dropped pairs."""
    r = rows.to(F8)[pos.long().clamp(min=0)]
    return r * (pos >= 0)[:, :, None]


# (and batches of several chunks of the sort, the last with more tokens to a chunk)
@pytest.mark.parametrize("T,d,E,k", SIZES + [(4097, 32, 896, 16), (131149, 32, 77, 2)])
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("bad", [False, True])
def test_dispatch(T, d, E, k, dtype, bad):
    r = routing()
    g, idx, _ = make(T, d, E, k, 1, bad)
    x = randn(g, T, d, dtype=dtype)
    rows, order = r.dispatch(x, idx, E)
    want = positions(idx, E)
    for got, ref, name in zip(order, want, order._fields):
        assert torch.equal(got.cpu().long(), ref), name
    for got, ref in zip(r.sort_pairs(idx, E), order):
        assert torch.equal(got, ref)
    pair = want[2].cuda()
    ref = x[pair.clamp(min=0) // k] * (pair >= 0)[:, None]
    assert torch.equal(rows, ref)


@pytest.mark.parametrize("T,d,E,k", SIZES)
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("out", DTS)
@pytest.mark.parametrize("bad", [False, True])
def test_dispatch_backward(T, d, E, k, dtype, out, bad):
    r = routing()
    g, idx, _ = make(T, d, E, k, 2, bad)
    order = r.sort_pairs(idx, E)
    drows = randn(g, T * k, d, dtype=dtype)
    if bad:   # what lies behind the last pair's row, or is its place, does not count
        drows[int(order.offsets[-1]):] = float("nan")
    dx = r.dispatch_backward(drows, order, out_dtype=out)
    v = gathered(drows.nan_to_num(0.0) if bad else drows, order.pair_pos)
    want = v.sum(1)
    within(dx, want, k * S24 * v.abs().sum(1) * 1.01 + step(want, out) * 1.01, "dx")


@pytest.mark.parametrize("T,d,E,k", SIZES)
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("out", DTS)
@pytest.mark.parametrize("bad,add", [(False, True), (True, False), (True, True)])
def test_collect(T, d, E, k, dtype, out, bad, add):
    r = routing()
    g, idx, w = make(T, d, E, k, 3, bad)
    order = r.sort_pairs(idx, E)
    rows = randn(g, T * k, d, dtype=dtype)
    a = randn(g, T, d, dtype=out) if add else None
    if bad:   # weight 0 skips its row, whatever that holds
        rows[int(order.offsets[-1]):] = float("inf")
        w[::2, 0] = 0.0
        p = order.pair_pos[::2, 0]
        rows[p[p >= 0].long()] = float("nan")
    y = r.collect(rows, order, w, add=a, out_dtype=out)
    v = gathered(torch.where(torch.isfinite(rows), rows, 0.0), order.pair_pos) * w.to(F8)[:, :, None]
    want, mag = v.sum(1), v.abs().sum(1)
    if add:
        want, mag = want + a.to(F8), mag + a.to(F8).abs()
    within(y, want, (k + 1) * S24 * mag * 1.01 + step(want, out) * 1.01, "y")


def test_collect_is_combine_for_fp32_rows():
    """The bits of k3moe_combine where both can be used."""
    r = routing()
    from mxfp4_routed_expert_gemv_amd import F32, k3moe_combine, make_shape
    g, idx, w = make(41, 7168, 896, 16, 4)
    order = r.sort_pairs(idx, 896)
    rows, add = randn(g, 41 * 16, 7168), randn(g, 41, 7168)
    y = r.collect(rows, order, w, add=add)
    want = torch.empty_like(y)
    k3moe_combine(make_shape(41, 7168, 32, 896, 16, 0, 0, F32, F32), rows, order.pair_pos, w, add, want)
    assert torch.equal(y, want)


@pytest.mark.parametrize("T,d,E,k", SIZES)
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("out", DTS)
@pytest.mark.parametrize("bad", [False, True])
def test_collect_backward(T, d, E, k, dtype, out, bad):
    r = routing()
    g, idx, w = make(T, d, E, k, 5, bad)
    order = r.sort_pairs(idx, E)
    rows, dy = randn(g, T * k, d, dtype=dtype), randn(g, T, d, dtype=out, std=0.1)
    drows, dw = r.collect_backward(dy, rows, order, w)
    n = int(order.offsets[-1])
    pair = order.sorted_pair.long()[:n]
    want = torch.zeros(T * k, d, dtype=F8, device="cuda")
    want[:n] = w.to(F8).view(-1)[pair][:, None] * dy.to(F8)[pair // k]
    within(drows, want, S24 * want.abs() + step(want, dtype) * 1.01, "drows")
    assert not drows[n:].any()
    v = gathered(rows, order.pair_pos) * dy.to(F8)[:, None, :]
    within(dw, v.sum(2), d * S24 * v.abs().sum(2) + 1e-300, "dw")
    only = r.collect_backward(dy, rows, order, w, need=(False, True))
    assert only[0] is None and torch.equal(only[1], dw)
    only = r.collect_backward(dy, rows, order, w, need=(True, False))
    assert only[1] is None and torch.equal(only[0], drows)


def route_case(T, d, E, k, router, dtype, bad, seed=6, skew=False):
    g, idx, _ = make(T, d, E, k, seed, bad, skew)
    logits = randn(g, T, E, std=2.0)
    at = idx.long().clamp(0, E - 1)
    chosen = logits.gather(1, at)
    if router == "softmax":
        w = torch.softmax(chosen, 1)
    else:
        w = torch.sigmoid(chosen)
        if router == "sigmoid_norm":
            w = w / w.sum(1, keepdim=True)
    return (randn(g, T, d, dtype=dtype), randn(g, E, d, dtype=torch.bfloat16, std=0.02), idx, w,
            randn(g, T, k, std=0.1), logits)


def route_reference(x, wr, idx, w, dw, logits, pos, router, T, d, E, k):
    there = pos >= 0
    w, dw = w.to(F8), dw.to(F8) * there
    at = idx.long().clamp(0, E - 1)
    few = (k + 12) * S24
    if router == "sigmoid":
        dl = dw * w * (1 - w)
        e_dl = few * (dw * w).abs()
    else:
        mean, mag = (w * dw).sum(1, keepdim=True), (w * dw).abs().sum(1, keepdim=True)
        dl, e_dl = w * (dw - mean), few * w * (dw.abs() + mag)
        if router == "sigmoid_norm":
            f = torch.sigmoid(-logits.to(F8).gather(1, at))
            dl, e_dl = dl * f, 2 * e_dl * f
    dl, e_dl = dl * there, e_dl * there
    wg = wr.to(F8)[at]
    dx = (dl[:, :, None] * wg).sum(1)
    dx_tol = ((e_dl + (k + 1) * S24 * dl.abs())[:, :, None] * wg.abs()).sum(1)
    flat = at.view(-1)
    tok = torch.arange(T * k, device="cuda") // k
    n = torch.bincount(flat, minlength=E).to(F8)[:, None]
    dwr = torch.zeros(E, d, dtype=F8, device="cuda")
    mag, err = dwr.clone(), dwr.clone()
    dwr.index_add_(0, flat, dl.view(-1, 1) * x.to(F8)[tok])
    mag.index_add_(0, flat, dl.abs().view(-1, 1) * x.to(F8)[tok].abs())
    err.index_add_(0, flat, e_dl.view(-1, 1) * x.to(F8)[tok].abs())
    return dx, dx_tol, dwr, (n + 1) * S24 * mag + err


@pytest.mark.parametrize("T,d,E,k", SIZES + [(3000, 96, 12, 4), (9000, 608, 30, 3)])
@pytest.mark.parametrize("router", ["softmax", "sigmoid", "sigmoid_norm"])
@pytest.mark.parametrize("dtype,out,bad", [(torch.bfloat16, torch.bfloat16, False),
                                           (torch.float32, torch.float32, True),
                                           (torch.bfloat16, torch.float32, True)])
def test_route_backward(T, d, E, k, router, dtype, out, bad):
    r = routing()
    x, wr, idx, w, dw, logits = route_case(T, d, E, k, router, dtype, bad, skew=T >= 3000)
    order = r.sort_pairs(idx, E)
    lg = logits if router == "sigmoid_norm" else None
    if bad:   # the weight gradient of a dropped pair does not count
        dw[order.pair_pos < 0] = float("nan")
    dx, dwr = r.route_backward(x, wr, idx, w, dw, order, router, lg, dw_dtype=out)
    want = route_reference(x, wr, idx, w, dw.nan_to_num(0.0), logits, order.pair_pos, router, T, d, E, k)
    within(dx, want[0], want[1] * 1.01 + step(want[0], dtype) * 1.01 + 1e-40, "dx")
    within(dwr, want[2], want[3] * 1.01 + step(want[2], out) * 1.01 + 1e-40, "dw_router")
    assert not dwr[order.counts == 0].any()
    only = r.route_backward(x, wr, idx, w, dw, order, router, lg, out, need=(False, True))
    assert only[0] is None and torch.equal(only[1], dwr)
    only = r.route_backward(x, wr, idx, w, dw, order, router, lg, out, need=(True, False))
    assert only[1] is None and torch.equal(only[0], dx)


def test_empty_batch():
    r = routing()
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    idx = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    rows, order = r.dispatch(x, idx, 16)
    assert rows.shape == (0, 256) and not order.counts.any() and not order.offsets.any()
    w = torch.empty(0, 4, device="cuda")
    assert r.collect(rows, order, w).shape == (0, 256)
    assert r.dispatch_backward(rows, order).shape == (0, 256)
    drows, dw = r.collect_backward(x, rows, order, w)
    assert drows.shape == (0, 256) and dw.shape == (0, 4)
    wr = torch.ones(16, 256, dtype=torch.bfloat16, device="cuda")
    dx, dwr = r.route_backward(x, wr, idx, w, w, order)
    assert dx.shape == (0, 256) and dwr.shape == (16, 256) and not dwr.any()


def test_bad_positions_touch_nothing():
    """Positions, ids and pairs outside their ranges are dropped, not followed."""
    r = routing()
    g, idx, w = make(40, 128, 8, 3, 7)
    order = r.sort_pairs(idx, 8)
    pos = order.pair_pos.clone()
    pos[::4, 1] = 1 << 30
    pos[1::4, 0] = -7
    pos[2::4, 2] = 120
    there = (pos >= 0) & (pos < 120)
    bad = order._replace(pair_pos=pos)
    rows = randn(g, 120, 128)
    y = r.collect(rows, bad, w)
    v = gathered(rows, torch.where(there, pos, -1)) * w.to(F8)[:, :, None]
    within(y, v.sum(1), 4 * S24 * v.abs().sum(1) * 1.01, "y")
    dy = randn(g, 40, 128)
    drows, dw = r.collect_backward(dy, rows, bad, w)
    assert not dw[~there].any()
    # offsets and pairs that make no sense give no sums, and end
    junk = order._replace(offsets=order.offsets * 1000 - 5, sorted_pair=order.sorted_pair - 60)
    wr = randn(g, 8, 128, dtype=torch.bfloat16)
    r.route_backward(rows[:40].contiguous(), wr, idx + 3, w, w, junk)
    torch.cuda.synchronize()


def test_one_more_device_check_and_types():
    r = routing()
    g, idx, w = make(8, 64, 4, 2, 8)
    x = randn(g, 8, 64)
    with pytest.raises(TypeError):
        r.dispatch(x.half(), idx, 4)
    with pytest.raises(TypeError):
        r.dispatch(x, idx.long(), 4)
    with pytest.raises(ValueError):
        r.dispatch(x[:, ::2], idx, 4)
    with pytest.raises(ValueError):
        r.dispatch(x, idx.cpu(), 4)
    with pytest.raises(ValueError):
        r.dispatch(x[:4].contiguous(), idx, 4)
    rows, order = r.dispatch(x, idx, 4)
    with pytest.raises(TypeError):
        r.collect(rows, order, w.double())
    with pytest.raises(TypeError):
        r.collect(rows, order, w, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        r.collect(rows, order, w, add=x.bfloat16(), out_dtype=torch.float32)
    with pytest.raises(ValueError):
        r.collect(rows[:-1], order, w)
    with pytest.raises(ValueError):
        r.route_backward(x, x[:4].bfloat16(), idx, w, w, order, router="top1")


# ------------------------------------------------------------- torch operations
def network(r, x, wr, experts, k, router, E):
    idx, w = r.route_tokens(x, wr, k, router)
    rows, order = r.dispatch_tokens(x, idx, E)
    at = order.offsets.tolist()
    ys = torch.cat([rows[at[e]:at[e + 1]] @ experts[e] for e in range(E)] + [rows[at[E]:]])
    return r.collect_tokens(ys, order, w, add=x), idx


@pytest.mark.parametrize("router", ["softmax", "sigmoid", "sigmoid_norm"])
def test_autograd_through_the_routing(router):
    """Route, sort, experts, collect in fp32: every gradient against the same network
    in 64 bits with the same choice.  The chain has about ten fp32 operations whose
    sums have at most T = 50 or d = 64 terms of unit size; 2^-24 * 64 * 10 of the
    largest gradient (and the router's weights are bf16, their gradient is rounded once)."""
    r = routing()
    T, d, E, k = 50, 64, 9, 3
    g = torch.Generator().manual_seed(11)
    x = randn(g, T, d).requires_grad_()
    wr = randn(g, E, d, dtype=torch.bfloat16, std=0.2).requires_grad_()
    experts = randn(g, E, d, d, std=0.1).requires_grad_()
    c = randn(g, T, d)
    y, idx = network(r, x, wr, experts, k, router, E)
    (y * c).sum().backward()

    X, WR, EX = (t.detach().to(F8).requires_grad_() for t in (x, wr, experts))
    l = (X @ WR.t()).gather(1, idx.long())
    w = torch.softmax(l, 1) if router == "softmax" else torch.sigmoid(l)
    if router == "sigmoid_norm":
        w = w / w.sum(1, keepdim=True)
    want = X + (w[:, :, None] * (X[:, None, None, :].float().to(F8) @ EX[idx.long()]).squeeze(2)).sum(1)
    (want * c.to(F8)).sum().backward()
    # X.float() above cuts nothing off (X holds fp32 values) but its gradient passes
    for got, ref, name, extra in ((y, want, "y", 0), (x.grad, X.grad, "dx", 0),
                                  (wr.grad, WR.grad, "dw_router", B), (experts.grad, EX.grad, "dexperts", 0)):
        tol = 640 * S24 * float(ref.abs().max()) + extra * ref.abs()
        within(got.detach(), ref.detach(), tol + torch.zeros_like(ref), name)


def test_gradients_against_differences():
    """dx of the whole network against central differences in 64 bits of its definition
    would repeat the test above; here the library's own forward is differenced.  With a
    step h the fp32 output's rounding gives 2^-24 |y| / h, the curvature h^2."""
    r = routing()
    T, d, E, k = 12, 32, 5, 2
    g = torch.Generator().manual_seed(13)   # (no choice is within 4 h of a tie)
    x = randn(g, T, d).requires_grad_()
    wr = randn(g, E, d, dtype=torch.bfloat16, std=0.2)
    c = randn(g, T, d)
    experts = randn(g, E, d, d, std=0.1)
    y, idx = network(r, x, wr, experts, k, "softmax", E)
    (y * c).sum().backward()
    v = randn(g, T, d)
    h = 2.0 ** -8

    def loss(s):
        out, at = network(r, (x.detach() + s * v), wr, experts, k, "softmax", E)
        assert torch.equal(at, idx)   # (the same choice on both sides)
        return float((out.to(F8) * c.to(F8)).sum())
    slope = (loss(h) - loss(-h)) / (2 * h)
    got = float((x.grad.to(F8) * v.to(F8)).sum())
    scale = float((y.detach().abs().to(F8) * c.abs().to(F8)).sum())
    tol = 64 * S24 * scale / h + 4 * h * h * scale
    log(f"  slope {slope:.6f}, gradient {got:.6f}, tolerance {tol:.2e}")
    assert abs(slope - got) <= tol


def test_another_stream_and_workspace():
    r = routing()
    g, idx, w = make(300, 512, 24, 6, 9)
    x = randn(g, 300, 512, dtype=torch.bfloat16)
    want, order = r.dispatch(x, idx, 24)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    st.wait_stream(torch.cuda.current_stream())
    rows, o2 = r.dispatch(x, idx, 24, workspace=ws, stream=st)
    y = r.collect(rows, o2, w, stream=st)
    st.synchronize()
    assert torch.equal(rows, want)
    assert torch.equal(y, r.collect(want, order, w))


def test_captured_and_replayed():
    """One graph of the forward and backward halves, replayed on new inputs with the
    program's own work between, every replay against the eager result."""
    r = routing()
    T, d, E, k = 600, 512, 24, 6
    g, idx, w = make(T, d, E, k, 10)
    x, dy = randn(g, T, d, dtype=torch.bfloat16), randn(g, T, d, dtype=torch.bfloat16)
    wr = randn(g, E, d, dtype=torch.bfloat16, std=0.02)

    def once():
        rows, order = r.dispatch(x, idx, E)
        y = r.collect(rows, order, w, add=x)
        drows, dw = r.collect_backward(dy, rows, order, w)
        dx = r.dispatch_backward(drows, order)
        return (y, dx, dw, *r.route_backward(x, wr, idx, w, dw, order))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        once()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = once()
    for i in range(4):
        _, idx2, w2 = make(T, d, E, k, 20 + i, bad=i == 2, skew=i == 3)
        idx.copy_(idx2)
        w.copy_(w2)
        x.copy_(randn(g, T, d, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b, name in zip(got, once(), ("y", "dx", "dw", "dx router", "dw_router")):
            assert torch.equal(a, b), (i, name)


def test_gradients_that_begin_inside_another_tensor():
    """What autograd hands a backward may be part of a larger tensor, at any element: the
    second half of a concatenation's gradient begins at 5 * 3 * 4 = 60 bytes here, rows'
    gradient at one element.  Moved, such a gradient gives the same bits."""
    r = routing()
    T, d, E, k = 5, 96, 7, 3
    g, *_ = make(T, d, E, k, 41)
    x = randn(g, T, d, dtype=torch.bfloat16).requires_grad_()
    wr = randn(g, E, d, dtype=torch.bfloat16, std=0.1).requires_grad_()
    dw = randn(g, 2 * T, k)
    idx, w = r.route_tokens(x, wr, k)
    want = torch.autograd.grad(w, (x, wr), dw[T:].clone(), retain_graph=True)
    both = torch.cat([torch.zeros(T, k, device="cuda"), w])
    got = torch.autograd.grad(both, (x, wr), dw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    def inside(t):   # t's values from the second element of a buffer on
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        at = buf[1:].view(t.shape)
        at.copy_(t)
        return at

    rows, order = r.dispatch_tokens(x, idx, E)
    up = randn(g, *rows.shape, dtype=rows.dtype)
    want, = torch.autograd.grad(rows, x, up, retain_graph=True)
    got, = torch.autograd.grad(rows, x, inside(up), retain_graph=True)
    assert torch.equal(got, want)
    leaf, wl = rows.detach().requires_grad_(), w.detach().requires_grad_()
    y = r.collect_tokens(leaf, order, wl)
    up = randn(g, T, d, dtype=y.dtype)
    want = torch.autograd.grad(y, (leaf, wl), up, retain_graph=True)
    got = torch.autograd.grad(y, (leaf, wl), inside(up))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
