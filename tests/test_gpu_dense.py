"""The dense operators on the GPU against their definitions in 64 bits.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value, an fp32
sum of n terms by at most n 2^-24 of the sum of the terms' magnitudes (and a
few more steps for each function of the sums); an output's bound adds the
roundings its inputs went through, each weighted with the magnitudes of what it
is multiplied with.  Beside that bound for every element, the error's norm over
a whole output of r roundings stays under 2^-8 sqrt(r) of the output's norm."""
import math

import pytest
import torch

from gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu

B, S24 = 2.0 ** -8, 2.0 ** -24
F8 = torch.float64


def normal(shape, seed, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def within(got, want, tol, roundings, name):
    assert got.shape == want.shape, (name, got.shape, want.shape)
    g = got.to(F8)
    assert torch.isfinite(g).all(), f"{name}: non-finite values"
    err = (g - want).abs()
    worst = float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0
    n = float(want.norm())
    rel = float(err.norm()) / n if n else 0.0
    log(f"  {name}: worst error {worst:.3f} of its bound, norm {rel:.2e}")
    assert worst <= 1.0, f"{name}: {worst:.3f} times its bound"
    if roundings:
        assert rel <= B * math.sqrt(roundings), f"{name}: norm of the error {rel:.2e}"


# ----------------------------------------------------- shared experts' training
class Ref:
    """Values and error bounds of the training pass, per element."""

    def __init__(self, x, w13, w2):
        self.x, self.w2 = x.to(F8), [w.to(F8) for w in w2]
        self.S, two_fs, d = w13.shape
        self.fs, self.T = two_fs // 2, x.shape[0]
        self.w13 = [w.to(F8) for w in w13]
        self.d = d

    def forward(self):
        gu, gu_tol, y, y_tol = [], [], 0, 0
        fs, few = self.fs, 16 * S24
        for w13, w2 in zip(self.w13, self.w2):
            p = self.x @ w13.t()
            acc = self.d * S24 * (self.x.abs() @ w13.abs().t())   # fp32 sum
            gu.append(p)
            gu_tol.append(acc + B * p.abs())
            g, u, ag, au = p[:, :fs], p[:, fs:], acc[:, :fs], acc[:, fs:]
            sil = g * torch.sigmoid(g)
            h = sil * u
            # |silu'| <= 1.1; the product of two fp32 values and its bf16 rounding
            e = 1.1 * ag * u.abs() + (sil.abs() + 1.1 * ag) * au + few * h.abs()
            e = e + B * (h.abs() + e)
            y = y + h @ w2.t()
            y_tol = y_tol + e @ w2.abs().t() + self.S * fs * S24 * (h.abs() + e) @ w2.abs().t()
        return y, y_tol, torch.stack(gu, 1), torch.stack(gu_tol, 1)

    def backward(self, gu, dy):
        fs, few, dy = self.fs, 16 * S24, dy.to(F8)
        dx, dx_tol, dw13, dw2 = 0, 0, [], []
        n_k = 2 * self.S * fs * S24
        for j, (w13, w2) in enumerate(zip(self.w13, self.w2)):
            g, u = gu[:, j, :fs].to(F8), gu[:, j, fs:].to(F8)
            s = torch.sigmoid(g)
            dh = dy @ w2
            dh_e = self.d * S24 * (dy.abs() @ w2.abs())
            sil, ds = g * s, s * (1 + g * (1 - s))
            # ds is a sum of two terms: its rounding is relative to their magnitudes
            ds_m = s + (g * s * (1 - s)).abs()
            p = torch.cat([dh * u * ds, dh * sil], 1)
            e = torch.cat([dh_e * (u * ds).abs() + few * (dh.abs() + dh_e) * u.abs() * ds_m,
                           dh_e * sil.abs() + few * (dh.abs() + dh_e) * sil.abs()], 1)
            e = e + B * (p.abs() + e)
            h = sil * u
            h_e = (B + few) * h.abs()
            dx = dx + p @ w13
            dx_tol = dx_tol + e @ w13.abs() + n_k * ((p.abs() + e) @ w13.abs())
            t_k = self.T * S24
            a = p.t() @ self.x
            dw13.append((a, e.t() @ self.x.abs() + t_k * ((p.abs() + e).t() @ self.x.abs())))
            b = dy.t() @ h
            dw2.append((b, dy.abs().t() @ h_e + t_k * (dy.abs().t() @ (h.abs() + h_e))))
        stack = lambda v, i: torch.stack([q[i] for q in v])  # noqa: E731
        return ((dx, dx_tol), (stack(dw13, 0), stack(dw13, 1)), (stack(dw2, 0), stack(dw2, 1)))


def rounded(want, tol, out=torch.bfloat16):
    return tol + (B * (want.abs() + tol) if out == torch.bfloat16 else S24 * want.abs())


def problem(T, d, fs, S, seed=1):
    std = 2.0 / math.sqrt(d)   # pre-activations of spread 2: the gate's curved part
    return (normal((T, d), seed), normal((S, 2 * fs, d), seed + 1, std),
            normal((S, d, fs), seed + 2, std))


SHARED = [(1, 32, 32, 1), (1, 256, 128, 2), (4, 256, 128, 1), (17, 96, 32, 3), (63, 64, 64, 8),
          (65, 288, 32, 8), (128, 128, 128, 1), (129, 160, 96, 2), (256, 512, 256, 1),
          (257, 480, 352, 2), (300, 544, 416, 2), (517, 1024, 512, 1), (1000, 32, 32, 1),
          (2100, 224, 160, 2), (640, 1536, 1024, 2), (1300, 2048, 1024, 2)]


@pytest.mark.parametrize("T,d,fs,S", SHARED)
def test_shared_train_and_backward(T, d, fs, S):
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.shared import shared_ffn_backward, shared_ffn_train
    x, w13, w2 = problem(T, d, fs, S)
    ref = Ref(x, w13, w2)
    y_want, y_tol, gu_want, gu_tol = ref.forward()
    for out in (torch.bfloat16, torch.float32):
        log(f"case T={T} d={d} fs={fs} S={S} {out}")
        y, gu = shared_ffn_train(x, w13, w2, out_dtype=out)
        torch.cuda.synchronize()
        within(y, y_want, rounded(y_want, y_tol, out), 2, "y")
        within(gu, gu_want, gu_tol, 1, "gu")
    dy = normal((T, d), 9, 0.1)
    got = shared_ffn_backward(x, gu, dy, w13, w2)
    torch.cuda.synchronize()
    for g, (want, tol), name in zip(got, ref.backward(gu, dy), ("dx", "dw13", "dw2")):
        within(g, want, rounded(want, tol), 2, name)
    # the same bits again, and one output at a time
    again = shared_ffn_backward(x, gu, dy, w13, w2)
    for i in range(3):
        one = shared_ffn_backward(x, gu, dy, w13, w2, need=[j == i for j in range(3)])
        assert torch.equal(again[i], got[i]) and torch.equal(one[i], got[i]), i
        assert [v is None for v in one] == [j != i for j in range(3)]


def test_shared_gradients_by_differences():
    """The backward against central differences of the 64-bit forward: a loss
    sum(c * y), moved along one random direction of each input."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.shared import shared_ffn
    T, d, fs, S = 33, 96, 64, 2
    x, w13, w2 = problem(T, d, fs, S, 20)
    c = normal((T, d), 30)
    ins = [t.clone().requires_grad_() for t in (x, w13, w2)]
    (shared_ffn(*ins) * c).sum().backward()

    def loss(a, b, w):
        return float((Ref(a, b, w).forward()[0] * c.to(F8)).sum())
    base = [t.to(F8) for t in (x, w13, w2)]
    for i, name in enumerate(("x", "w13", "w2")):
        v = normal(base[i].shape, 40 + i, dtype=torch.float64)
        step = 1e-5
        hi, lo = ([b + (s * step * v if j == i else 0) for j, b in enumerate(base)] for s in (1, -1))
        want = (loss(*hi) - loss(*lo)) / (2 * step)
        grad = ins[i].grad.to(F8)
        got = float((grad * v).sum())
        # along a random direction the elements' independent errors (at most
        # 4 roundings each: gu, dgu or h, and the output) add up as their norm
        tol = 4 * 2 * B * float(grad.norm())
        log(f"  {name}: {got:.5g} for {want:.5g} (allowed {tol:.2g})")
        assert abs(got - want) <= tol, name


def test_shared_empty_batch_and_bad_tokens():
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.shared import shared_ffn_backward, shared_ffn_train
    x, w13, w2 = problem(70, 96, 64, 2, 50)
    y, gu = shared_ffn_train(x[:0], w13, w2)
    assert y.shape == (0, 96) and gu.shape == (0, 2, 128)
    dx, dw13, dw2 = shared_ffn_backward(x[:0], gu, x[:0], w13, w2)
    assert dx.shape == (0, 96) and not dw13.any() and not dw2.any()
    # a token of infinities or NaN reaches its own rows of y and dx only, and
    # extreme gates stay finite
    good, gu_good = shared_ffn_train(x, w13, w2)
    bad = x.clone()
    bad[5], bad[68, 3] = float("inf"), float("nan")
    y, gu = shared_ffn_train(bad, w13, w2)
    rows = torch.ones(70, dtype=torch.bool)
    rows[[5, 68]] = False
    assert torch.equal(y[rows.cuda()], good[rows.cuda()])
    assert not torch.isfinite(y[~rows.cuda()]).all(1).any()
    dy = normal((70, 96), 51)
    dx_good = shared_ffn_backward(x, gu_good, dy, w13, w2)[0]
    dx = shared_ffn_backward(bad, gu, dy, w13, w2)[0]
    assert torch.equal(dx[rows.cuda()], dx_good[rows.cuda()])
    far = gu_good.clone()
    far[:, :, :64] = torch.tensor([-3e38, -200.0, -89.0, 89.0, 3e38, 0.0, -0.0, 1.0] * 8)
    dw13 = shared_ffn_backward(x, far, dy, w13, w2)[1]
    # row f of dW13 sums feature f's dg (or, fs further, du) over the tokens.  dg
    # is finite at every gate here (its factor is sigmoid(g) (1 + g (1 -
    # sigmoid(g))), 1 at 3e38); du = dh silu(g) reaches 3e38 |dh| at the gate
    # 3e38, beyond bf16's and fp32's range, and nowhere else
    assert torch.isfinite(dw13[:, :64]).all()
    over = torch.arange(64) % 8 == 4
    assert torch.isfinite(dw13[:, 64:][:, ~over.cuda()]).all()


def test_shared_rows_behind_the_batch_stay():
    """Outputs longer than the batch keep what was behind it."""
    require_gpu()
    import mxfp4_routed_expert_gemv_amd as k3
    from mxfp4_routed_expert_gemv_amd import shared
    T, d, fs, S = 37, 96, 32, 2
    x, w13, w2 = problem(T, d, fs, S, 60)
    shape, bank, nbytes, _ = shared._problem(x, w13, w2, torch.bfloat16, k3.OP_SHARED_BACKWARD)
    y = torch.full((T + 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    gu = torch.full((T + 3, S, 2 * fs), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = y.clone()
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    k3.k3moe_shared_ffn_train(shape, bank, x, gu, y, ws)
    k3.k3moe_shared_ffn_backward(shape, bank, x, gu, x, dx, None, None, ws)
    torch.cuda.synchronize()
    assert (y[T:] == 7).all() and (gu[T:] == 7).all() and (dx[T:] == 7).all()
    assert torch.equal(y[:T], shared.shared_ffn_train(x, w13, w2)[0])


# ------------------------------------------------------- 4-bit weights
def w4_problem(T, n, k, group, zero, dtype, seed=3):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8).cuda()
    scale = (torch.rand((n, k // group), generator=g) * 0.1 + 0.01).bfloat16().cuda()
    z = torch.randint(0, 16, (n, k // group), generator=g, dtype=torch.uint8).cuda() if zero else None
    return normal((T, k), seed + 1, dtype=dtype), codes, scale, z


def w4_dense(codes, scale, zero):
    n, half = codes.shape
    q = torch.stack([codes & 15, codes >> 4], -1).view(n, scale.shape[1], -1).to(F8)
    z = 8.0 if zero is None else zero.to(F8)[..., None]
    s = scale.to(F8)[..., None]
    # the weights, and the magnitudes that enter the kernel's sums: (16 + q) and (16 + z)
    return ((q - z) * s).view(n, -1), ((32 + q + z) * s.abs()).view(n, -1)


def w4_bounds(x, codes, scale, zero):
    w, m = w4_dense(codes, scale, zero)
    x = x.to(F8)
    # an element's terms meet at most 128 / 32 steps of 32 within a group, the
    # groups of a wave's slice and the waves: k / 32 + 64 roundings cover them,
    # and three times that the three parts of an fp32 activation
    steps = 3 * (x.shape[1] // 32 + 64)
    return x @ w.t(), steps * S24 * (x.abs() @ m.t())


W4 = [(1, 64, 128, 128, False), (1, 17, 32, 32, True), (2, 100, 96, 32, False),
      (5, 33, 192, 64, True), (6, 258, 160, 32, False), (15, 2, 640, 128, True),
      (16, 130, 1024, 128, False), (17, 96, 1088, 64, True), (21, 66, 256, 256, False),
      (22, 1000, 512, 512, True), (33, 98, 2048, 128, True), (64, 514, 4096, 32, True),
      (65, 64, 384, 128, False), (131, 40, 224, 32, True), (1, 2050, 7168, 128, True),
      (3, 7168, 2048, 64, False), (300, 130, 640, 64, True), (257, 66, 1280, 128, False)]


@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,n,k,group,zero", W4)
def test_w4_products(T, n, k, group, zero, xd):
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.w4 import w4_glu, w4_linear
    x, codes, scale, z = w4_problem(T, n, k, group, zero, xd)
    want, tol = w4_bounds(x, codes, scale, z)
    for out in (torch.float32, torch.bfloat16):
        log(f"case T={T} n={n} k={k} group={group} zero={zero} {xd} -> {out}")
        got = w4_linear(x, codes, scale, z, out_dtype=out)
        torch.cuda.synchronize()
        within(got, want, rounded(want, tol, out), 0, "linear")
        if n % 2 == 0:
            f = n // 2
            g, u, ge, ue = want[:, :f], want[:, f:], tol[:, :f], tol[:, f:]
            sil = g * torch.sigmoid(g)
            h = sil * u
            e = 1.1 * ge * u.abs() + (sil.abs() + 1.1 * ge) * ue + 16 * S24 * h.abs()
            got = w4_glu(x, codes, scale, z, out_dtype=out)
            torch.cuda.synchronize()
            within(got, h, rounded(h, e, out), 0, "glu")


def test_w4_tokens_do_not_depend_on_the_batch():
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.w4 import w4_linear
    x, codes, scale, z = w4_problem(40, 96, 1024, 64, True, torch.bfloat16, 11)
    want, tol = w4_bounds(x, codes, scale, z)
    for T in (1, 2, 16, 17, 40):
        got = w4_linear(x[:T].contiguous(), codes, scale, z, out_dtype=torch.float32)
        assert ((got.to(F8) - want[:T]).abs() <= rounded(want[:T], tol[:T], torch.float32)).all(), T


@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
def test_w4_special_values(xd):
    """Infinities and NaN in x and scale give what the definition gives: an
    infinity times a weight of its sign, NaN where the weight is zero."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.w4 import w4_linear
    x, codes, scale, z = w4_problem(7, 48, 512, 128, True, xd, 21)
    codes[0, :] = 0xFF   # rows of one sign: an infinity keeps it
    codes[1, :] = 0x00
    z[:] = 8
    codes[2, 5] = 0x88   # a zero weight against the infinity
    x[1, 10] = float("inf")
    x[2, 10] = float("-inf")
    x[3, 300] = float("nan")
    x[4, 7] = torch.finfo(xd).max    # finite, but 16 times it is not
    x[4, 8:] = 0
    scale[5, 2] = float("inf")
    scale[6, 1] = float("nan")
    got = w4_linear(x, codes, scale, z, out_dtype=torch.float32).cpu()
    w, _ = w4_dense(codes.cpu(), scale.cpu(), z.cpu())
    want = torch.zeros(7, 48, dtype=F8)
    for t in range(7):
        want[t] = (x[t].cpu().to(F8) * w).sum(1)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert inf.any() and torch.equal(got[inf].to(F8), want[inf])
    # (a sum past fp32's range is an infinity in fp32)
    fine = torch.isfinite(want) & (want.abs() < 3e38)
    mag = (x.cpu().to(F8).abs().nan_to_num(0, 0, 0) @ w.abs().nan_to_num(0, 0, 0).t())
    assert ((got.to(F8) - want).abs()[fine] <= 1e-4 * mag[fine]).all()


# ------------------------------------------------------- gradients' norm
def grad_list(sizes, dtypes, odd, seed=5, std=0.01):
    out = []
    for i, (n, dt) in enumerate(zip(sizes, dtypes)):
        flat = normal((n + odd,), seed + i, std, dt)
        out.append(flat[odd:])
    return out


BF, F4 = torch.bfloat16, torch.float32
GRADS = [([1], [BF], 0), ([7], [F4], 1), ([8, 9, 0, 16383], [BF, F4, BF, BF], 1),
         ([16384, 16385, 1, 100_003], [F4, BF, F4, BF], 3), ([5_000_001], [BF], 1),
         ([40_000_000], [F4], 0), ([3 + 17 * i for i in range(300)], [BF, F4] * 150, 1)]


def norm64(ts):
    return math.sqrt(math.fsum(float((t.to(F8) ** 2).sum()) for t in ts))


@pytest.mark.parametrize("sizes,dtypes,odd", GRADS)
def test_grad_norm_and_clip(sizes, dtypes, odd):
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.grads import clip_grads, grad_norm
    ts = grad_list(sizes, dtypes, odd)
    want = norm64(ts)
    # fp64 sums: the rounding to fp32 alone is left
    assert abs(float(grad_norm(ts)) - want) <= S24 * want * 1.001
    for max_norm in (want / 3, want * 3):
        factor = min(1.0, max_norm / want)
        outs = [torch.full((t.numel() + 2,), 9.0, dtype=dt, device="cuda")[1:-1]
                for t, dt in zip(ts, dtypes[1:] + dtypes[:1])]
        before = [t.clone() for t in ts]
        log(f"case {len(sizes)} tensors, {sum(sizes)} elements, factor {factor:.3f}")
        got = clip_grads(ts, max_norm, out=outs)
        assert abs(float(got) - want) <= S24 * want * 1.001
        for t, b, o in zip(ts, before, outs):
            exact = t.to(F8) * factor
            # the factor's rounding, the product's and the output's
            eps = 2 * S24 + (B if o.dtype == BF else 0.0)
            assert torch.equal(t, b)
            assert ((o.to(F8) - exact).abs() <= eps * exact.abs() * 1.001).all()
            if factor == 1.0:
                assert torch.equal(o, t.to(o.dtype))
        assert torch.equal(clip_grads(ts, max_norm), got)   # in place
        for t, b in zip(ts, before):
            exact = b.to(F8) * factor
            eps = 2 * S24 + (B if t.dtype == BF else 0.0)
            assert ((t.to(F8) - exact).abs() <= eps * exact.abs() * 1.001).all()
            t.copy_(b)


def test_grad_extremes():
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.grads import clip_grads, grad_norm
    big = [torch.full((1000,), 1e30, device="cuda"), torch.full((3,), 3e38, device="cuda").bfloat16()]
    # three elements of 3e38 have the norm sqrt(3) 3e38 = 5.2e38, past fp32's 3.4e38;
    # the list's first has 1e30 sqrt(1000) = 3.2e31, inside it, though not its square
    assert float(grad_norm(big)) == float("inf")
    assert abs(float(grad_norm(big[:1])) / norm64(big[:1]) - 1) <= S24 * 1.001
    small = [torch.full((1001,), 1e-42, device="cuda")]   # squares far below fp32's range
    assert abs(float(grad_norm(small)) - norm64(small)) <= 2.0 ** -149
    zero = [torch.zeros(10, device="cuda")]
    assert float(clip_grads(zero, 1.0)) == 0.0 and not zero[0].any()
    # a norm of zero allowed: everything becomes zero
    ts = grad_list([50, 60], [BF, F4], 0)
    assert float(clip_grads(ts, 0.0)) > 0 and not any(t.any() for t in ts)
    for bad in (float("inf"), float("nan"), float("-inf")):
        ts = grad_list([50, 60_000], [BF, F4], 0)
        ts[1][777] = bad
        before = [t.clone() for t in ts]
        got = float(clip_grads(ts, 1e-3))
        assert not math.isfinite(got) and math.isnan(got) == math.isnan(bad)
        assert all(torch.equal(t.nan_to_num(5), b.nan_to_num(5)) for t, b in zip(ts, before))
    # a norm past fp32's range, of finite gradients, still clips
    huge = [torch.full((4,), 3e38, device="cuda")]
    assert float(clip_grads(huge, 1.0)) == float("inf")
    assert torch.allclose(huge[0], torch.full_like(huge[0], 0.5), rtol=1e-6)
    # the same tensor twice counts twice
    t = grad_list([100], [F4], 0)[0]
    assert abs(float(grad_norm([t, t])) - norm64([t, t])) <= S24 * norm64([t, t]) * 1.001


# ------------------------------------------------------- used together
def test_a_training_step_then_serving_in_4_bits():
    """Forward, loss, backward, clipping and an update of the shared experts, the
    updated block then served from 4-bit weights."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.grads import clip_grads
    from mxfp4_routed_expert_gemv_amd.shared import shared_ffn
    from mxfp4_routed_expert_gemv_amd.w4 import w4_glu, w4_linear
    T, d, fs, S = 96, 256, 128, 2
    x, w13, w2 = problem(T, d, fs, S, 70)
    target = normal((T, d), 75)
    p13, p2 = w13.clone().requires_grad_(), w2.clone().requires_grad_()
    y = shared_ffn(x, p13, p2)
    loss = ((y - target).float() ** 2).mean()
    loss.backward()
    ref = Ref(x, w13, w2)
    y64 = ref.forward()[0]
    gu = torch.stack([x.to(F8) @ w.to(F8).t() for w in w13], 1)
    dy64 = 2 * (y64 - target.to(F8)) / y64.numel()
    (dx, _), (dw13, _), (dw2, _) = ref.backward(gu, dy64)
    for got, want in ((p13.grad, dw13), (p2.grad, dw2)):
        # roundings on the way: y, the loss's gradient, gu, dgu or h, the output
        assert float((got.to(F8) - want).norm()) <= 5 * B * float(want.norm())
    before = norm64([p13.grad, p2.grad])
    outs = [torch.empty_like(p, dtype=torch.float32) for p in (p13, p2)]
    norm = clip_grads([p13.grad, p2.grad], before / 2, out=outs)
    assert abs(float(norm) - before) <= 2 * S24 * before
    assert abs(norm64(outs) - before / 2) <= 4 * S24 * before
    with torch.no_grad():
        for p, g in zip((p13, p2), outs):
            p -= (0.5 * g).to(p.dtype)

    def quantise(w, group=64):
        v = w.float().view(w.shape[0], -1, group)
        s = (v.abs().amax(-1) / 7).clamp(min=1e-8).bfloat16()
        q = (v / s.float()[..., None]).round().clamp(-8, 7).add(8).to(torch.uint8).view(w.shape)
        return (q[:, 0::2] | q[:, 1::2] << 4).contiguous(), s
    # both experts side by side: all gates, then all ups
    w13f = torch.cat([p13.detach()[:, :fs].reshape(S * fs, d), p13.detach()[:, fs:].reshape(S * fs, d)])
    w2f = p2.detach().transpose(0, 1).reshape(d, S * fs)
    (c13, s13), (c2, s2) = quantise(w13f), quantise(w2f.contiguous())
    one = x[:1].contiguous()
    h = w4_glu(one, c13, s13)
    out = w4_linear(h, c2, s2, out_dtype=torch.float32)
    torch.cuda.synchronize()
    g64 = one.to(F8) @ w4_dense(c13, s13, None)[0].t()
    h64 = g64[:, :S * fs] * torch.sigmoid(g64[:, :S * fs]) * g64[:, S * fs:]
    w64 = w4_dense(c2, s2, None)[0]
    assert float((out.to(F8) - h64 @ w64.t()).norm()) <= 2 * B * float((h64.abs() @ w64.abs().t()).norm())


def test_captured_and_replayed_on_other_streams():
    """A captured step (training pass, norm and clip, 4-bit products) replayed
    with new inputs between eager work; and eager calls on a side stream."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.grads import clip_grads
    from mxfp4_routed_expert_gemv_amd.shared import shared_ffn_backward, shared_ffn_train
    from mxfp4_routed_expert_gemv_amd.w4 import w4_linear
    T, d, fs, S = 45, 160, 96, 2
    x, w13, w2 = problem(T, d, fs, S, 80)
    wx, codes, scale, z = w4_problem(3, 64, 256, 64, True, torch.float32, 85)

    def step():
        y, gu = shared_ffn_train(x, w13, w2)
        grads = shared_ffn_backward(x, gu, y, w13, w2)
        outs = [torch.empty_like(g, dtype=torch.float32) for g in grads]
        norm = clip_grads(grads, 0.5, out=outs)
        return [y, gu, *grads, norm, *outs, w4_linear(wx, codes, scale, z)]
    eager = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        x.copy_(normal((T, d), 90 + i))
        wx.copy_(normal((3, 256), 95 + i, dtype=torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i


# ------------------------------------------------------- where forms change
@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("T", [4, 8, 9, 16, 32, 64, 70, 128, 200])
def test_w4_at_the_token_counts_where_the_form_changes(T, group, xd):
    """Both sides of each change of kernel, with a last block and a last weight
    row inside a tile and a contraction whose split pieces are uneven."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.w4 import w4_linear
    n, k = 131, 5 * 256 + group
    for t in (T, T + 1):
        x, codes, scale, z = w4_problem(t, n, k, group, group != 64, xd, 100 + t)
        want, tol = w4_bounds(x, codes, scale, z)
        log(f"case T={t} group={group} {xd}")
        room = torch.full((t * n + 64,), 7.0, device="cuda")   # (out: 16-byte aligned)
        out = room[32:-32].view(t, n)
        w4_linear(x, codes, scale, z, out=out)
        torch.cuda.synchronize()
        within(out, want, rounded(want, tol, torch.float32), 0, "linear")
        assert (room[:32] == 7).all() and (room[-32:] == 7).all()


@pytest.mark.parametrize("n", [8192, 8224])
def test_w4_on_both_sides_of_one_round_of_workgroups(n):
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.w4 import w4_glu
    x, codes, scale, z = w4_problem(40, n, 512, 128, True, torch.bfloat16, 120)
    want, tol = w4_bounds(x, codes, scale, z)
    f = n // 2
    g, u, ge, ue = want[:, :f], want[:, f:], tol[:, :f], tol[:, f:]
    sil = g * torch.sigmoid(g)
    h = sil * u
    e = 1.1 * ge * u.abs() + (sil.abs() + 1.1 * ge) * ue + 16 * S24 * h.abs()
    got = w4_glu(x, codes, scale, z)
    torch.cuda.synchronize()
    within(got, h, rounded(h, e), 0, "glu")


@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,n,k", [(20, 48, 512), (50, 48, 512), (70, 48, 768), (140, 260, 768)])
def test_w4_special_values_in_larger_batches(T, n, k, xd):
    """As for few tokens: a value that is not finite reaches its own token's (or
    weight row's) outputs alone."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.w4 import w4_linear
    x, codes, scale, z = w4_problem(T, n, k, 128, True, xd, 130)
    codes[0, :], codes[1, :] = 0xFF, 0x00
    z[:] = 8
    x[T - 1, 10] = float("inf")
    x[T - 2, k - 1] = float("-inf")
    x[0, 300] = float("nan")
    x[17, 7] = torch.finfo(xd).max    # finite, but 16 times it is not
    x[17, 8:] = 0
    scale[n - 1, 2] = float("inf")
    scale[6, 1] = float("nan")
    got = w4_linear(x, codes, scale, z, out_dtype=torch.float32).cpu()
    w, _ = w4_dense(codes.cpu(), scale.cpu(), z.cpu())
    want = torch.stack([(row.to(F8) * w).sum(1) for row in x.cpu()])
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert inf.any() and torch.equal(got[inf].to(F8), want[inf])
    fine = torch.isfinite(want) & (want.abs() < 3e38)
    mag = (x.cpu().to(F8).abs().nan_to_num(0, 0, 0) @ w.abs().nan_to_num(0, 0, 0).t())
    assert ((got.to(F8) - want).abs()[fine] <= 1e-4 * mag[fine]).all()


@pytest.mark.parametrize("dt", [BF, F4])
def test_clip_with_the_norm_joined_in_a_launch_of_its_own(dt):
    """A list of so many pieces that the scaling does not join them itself."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.grads import clip_grads
    ts = grad_list([60_000_000] + [129 + i for i in range(250)], [dt] * 251, 1, 140)
    want = norm64(ts)
    outs = [torch.empty_like(t) for t in ts]
    got = clip_grads(ts, want / 4, out=outs)
    assert abs(float(got) - want) <= S24 * want * 1.001
    for t, o in zip(ts, outs):
        exact = t.to(F8) * 0.25   # the factor's, the product's and the output's rounding
        eps = 3 * S24 + (B if dt == BF else 0.0)
        assert ((o.to(F8) - exact).abs() <= eps * exact.abs() * 1.001).all()


def test_a_given_stream_and_workspaces_of_one_graph_beside_another():
    """Calls on a stream that is not current, and two graphs whose calls were given
    one workspace, replayed in turn."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.grads import clip_grads, grad_norm
    from mxfp4_routed_expert_gemv_amd.shared import shared_ffn_backward, shared_ffn_train
    from mxfp4_routed_expert_gemv_amd.w4 import w4_glu, w4_linear
    T, d, fs, S = 70, 256, 64, 1
    x, w13, w2 = problem(T, d, fs, S, 150)
    wx, codes, scale, z = w4_problem(T, 64, 2048, 64, True, torch.bfloat16, 155)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def step(workspace=None, stream=None):
        y, gu = shared_ffn_train(x, w13, w2, workspace=workspace, stream=stream)
        grads = shared_ffn_backward(x, gu, y, w13, w2, workspace=workspace, stream=stream)
        more = [w4_linear(wx, codes, scale, z, workspace=workspace, stream=stream),
                w4_glu(wx, codes, scale, z, workspace=workspace, stream=stream)]
        outs = [torch.empty_like(g) for g in grads]
        return [y, gu, *grads, *more, grad_norm(grads, stream=stream),
                clip_grads(grads, 0.1, out=outs, stream=stream), *outs]

    def same(a, b):
        return all(torch.equal(p, q) for p, q in zip(a, b))
    eager = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(stream=side)
    side.synchronize()
    assert same(eager, other)
    graphs, held = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(step(ws))
        graphs.append(g)
    for i in range(3):
        x.copy_(normal((T, d), 160 + i))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert same(held[0], want) and same(held[1], want), i


# tokens, d, fs, experts: every tile of each product, with its contraction whole and in
# pieces, batches and features that end inside a tile
TILES = [(65, 2048, 832, 2), (66, 3104, 2048, 1), (67, 2016, 1568, 2), (132, 3136, 1408, 3),
         (131, 3392, 1472, 3), (1, 2048, 1984, 2), (402, 256, 1760, 2), (261, 256, 1856, 3),
         (769, 256, 1280, 3), (662, 256, 1824, 3), (848, 3488, 128, 1), (1061, 3616, 128, 1),
         (2, 2240, 960, 3), (3, 2912, 1440, 3)]


@pytest.mark.parametrize("T,d,fs,S", TILES)
def test_shared_tiles_and_splits(T, d, fs, S):
    test_shared_train_and_backward(T, d, fs, S)


@pytest.mark.parametrize("T,d,fs,S", [(1, 256, 128, 1), (2, 64, 32, 3), (4, 256, 128, 1), (15, 512, 64, 3),
                                      (16, 320, 256, 2), (1, 2048, 1984, 2), (3, 4096, 512, 1)])
def test_shared_values_of_few_tokens_keep_16_bits(T, d, fs, S, monkeypatch):
    """Up to 16 tokens h, dg and du are two bf16 parts: the first, cut off, leaves 2^-7
    of a value, the second 2^-8 of that.  So an fp32 y is off by 2^-15 of its terms,
    and a bf16 output, as its rounding to the nearest moves by no more than its argument
    does, by the exact value's own rounding and twice such a bound."""
    require_gpu()
    import sys
    from mxfp4_routed_expert_gemv_amd.shared import shared_ffn_backward, shared_ffn_train
    x, w13, w2 = problem(T, d, fs, S, 170)
    y, gu = shared_ffn_train(x, w13, w2, out_dtype=torch.float32)
    dy = normal((T, d), 175, 0.1)
    grads = shared_ffn_backward(x, gu, dy, w13, w2)
    torch.cuda.synchronize()
    ref = Ref(x, w13, w2)
    monkeypatch.setattr(sys.modules[__name__], "B", 2.0 ** -15)
    want, tol = ref.forward()[:2]
    back = ref.backward(gu, dy)
    monkeypatch.undo()
    within(y, want, rounded(want, tol, torch.float32), 0, "y")
    for g, (want, tol), name in zip(grads, back, ("dx", "dw13", "dw2")):
        own = float((want.bfloat16().to(F8) - want).norm())
        err = float((g.to(F8) - want).norm())
        log(f"  {name}: error {err:.3e}, its rounding alone {own:.3e}, parts {float(tol.norm()):.3e}")
        assert err <= own + 2 * float(tol.norm()), name


@pytest.mark.parametrize("T,d,fs,S", [(10001, 7168, 2048, 2), (16385, 4096, 1504, 3), (12289, 6144, 4096, 1)])
def test_shared_weight_gradients_of_large_batches(T, d, fs, S):
    """Both weight gradients in one launch, the rows of dw2 behind its full rounds in
    another: each row and column written, alone (in launches of their own) the same
    bits, and sampled columns as defined."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.shared import shared_ffn_backward
    x, w13, w2 = problem(T, d, fs, S, 180)
    gu, dy = normal((T, S, 2 * fs), 185), normal((T, d), 186, 0.1)
    dx, dw13, dw2 = shared_ffn_backward(x, gu, dy, w13, w2)
    for i, got in ((0, dx), (1, dw13), (2, dw2)):
        one = shared_ffn_backward(x, gu, dy, w13, w2, need=[j == i for j in range(3)])[i]
        assert torch.equal(one, got), i
    cols = torch.cat([torch.arange(0, fs, 301), torch.tensor([fs - 1])]).cuda()
    few = S24 * T
    for j in range(S):
        g, u = gu[:, j, cols].to(F8), gu[:, j, fs + cols].to(F8)
        h = g * torch.sigmoid(g) * u
        want = dy.to(F8).t() @ h
        tol = (B + 17 * S24 + few) * (dy.to(F8).abs().t() @ h.abs())
        within(dw2[j][:, cols], want, rounded(want, tol), 2, f"dw2 of expert {j}")
        dh = dy.to(F8) @ w2[j].to(F8)[:, cols]
        du = dh * g * torch.sigmoid(g)
        want = du.t() @ x.to(F8)
        dh_e = d * S24 * (dy.to(F8).abs() @ w2[j].to(F8)[:, cols].abs())
        e = B * du.abs() + 2 * (dh_e + 16 * S24 * dh.abs()) * (g * torch.sigmoid(g)).abs()
        tol = (e + few * (du.abs() + e)).t() @ x.to(F8).abs()
        within(dw13[j][fs + cols], want, rounded(want, tol), 2, f"dw13 (up) of expert {j}")


@pytest.mark.parametrize("T", [3, 16, 17, 40])
def test_shared_infinite_gradients_and_weights(T):
    """An infinite dy or weight gives infinities and NaN where the formulas do, with
    one part to a value or two, and leaves what it does not enter."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.shared import shared_ffn_backward, shared_ffn_train
    d, fs, S = 256, 96, 2
    x, w13, w2 = problem(T, d, fs, S, 190)
    y, gu = shared_ffn_train(x, w13, w2)
    dy = normal((T, d), 195, 0.1)
    fine = shared_ffn_backward(x, gu, dy, w13, w2)
    dy[2, 7] = float("inf")
    dx, dw13, dw2 = shared_ffn_backward(x, gu, dy, w13, w2)
    torch.cuda.synchronize()

    def same_kind(got, want, name):
        assert torch.equal(torch.isnan(got), torch.isnan(want)), name
        inf = torch.isinf(want)
        assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf].to(F8), want[inf]), name
    keep = torch.arange(T) != 2
    assert torch.equal(dx[keep], fine[0][keep]) and not torch.isfinite(dx[2]).any()
    for j in range(S):
        g, u = gu[:, j, :fs].to(F8).cpu(), gu[:, j, fs:].to(F8).cpu()
        h = g * torch.sigmoid(g) * u
        same_kind(dw2[j].cpu(), sum(dy[t].to(F8).cpu()[:, None] * h[t] for t in range(T)), "dw2")
        assert torch.isinf(dw2[j][7]).all() and torch.isinf(dw13[j]).all()
    w2[1, 9, 5] = float("-inf")
    got = shared_ffn_train(x, w13, w2)[0]
    torch.cuda.synchronize()
    g, u = (x.to(F8) @ w.to(F8).t() for w in (w13[1, 5:6], w13[1, fs + 5:fs + 6]))
    want = torch.where((g * u)[:, 0] > 0, -math.inf, math.inf)   # silu has its argument's sign
    assert torch.equal(got[:, 9].to(F8), want)
    others = torch.arange(d) != 9
    assert torch.equal(got[:, others], y[:, others])


@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,zero", [(1, 1280, True), (3, 4096, False), (7, 128, True), (12, 2176, True),
                                      (30, 1152, False), (50, 1280, True), (90, 1152, True), (300, 640, False)])
def test_w4_groups_of_32_in_whole_blocks(T, k, zero, xd):
    """Contractions that are a multiple of 128, whose four scales a block are copied
    together; and what the gated form's two halves read."""
    require_gpu()
    test_w4_products(T, 134, k, 32, zero, xd)


@pytest.mark.parametrize("T,d,fs,S", [(1101, 3520, 768, 2), (2500, 1536, 1024, 1), (7190, 1088, 128, 1),
                                      (3001, 2560, 1600, 2)])
def test_shared_gradients_in_one_launch(T, d, fs, S):
    """Gradients whose tiles share a launch, with dx on smaller tiles than the
    weights' and on the same; alone they come from launches of their own."""
    test_shared_train_and_backward(T, d, fs, S)
