"""The dense operators on the GPU where a call is at the edge of what the header
allows.  Tolerances as in test_gpu_dense: half a step of a type is eps / 2 of a
value (bf16 2^-8, fp32 2^-24)."""
import math

import pytest
import torch

from gpu_util import log, require_gpu
from test_gpu_dense import B, F8, S24

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value,count,max_norm", [
    (3e38, 4, 1e-3), (3e38, 4, 1e-7), (3e38, 70_001, 1.0), (3e38, 16_411, 1e-30), (1e25, 9, 1e-14),
    (2e38, 3, 1e-1)])
def test_clip_by_a_factor_below_fp32s_normal_range(value, count, max_norm, dt, out):
    """max_norm / norm under 2^-126 is no normal fp32 number, but the clipped gradients
    are: each is off by its own rounding to fp32 (the factor is fp64, off by a few
    2^-53), a bf16 one by bf16's on top, and by max_norm's, which enters the call as a C
    float: m (1 + a) g / norm (1 + b) with |a|, |b| <= 2^-24."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.grads import clip_grads
    g = torch.full((count,), value, device="cuda").to(dt)
    g[1] = -g[1] / 3
    g[2] = g[2] / 1024
    norm = math.sqrt(math.fsum((g.to(F8) ** 2).tolist()))
    factor = max_norm / norm
    assert factor < 2.0 ** -126
    want = g.to(F8) * factor
    eps = 2 * S24 * 1.001 + (B if out == torch.bfloat16 else 0.0)
    for name, outs in (("into", [torch.empty_like(g, dtype=out)]), ("in place", None)):
        if outs is None and dt != out:
            continue
        clip_grads([g], max_norm, out=outs)
        torch.cuda.synchronize()
        got = (outs or [g])[0].to(F8)
        worst = float(((got - want).abs() / want.abs()).max())
        log(f"  {value:g} x {count}, max_norm {max_norm:g}, {dt} -> {out} {name}: factor {factor:.3g}, worst {worst:.3g}")
        # (smallest outputs here: 1e-30 / sqrt(16411) / 1024 = 7.6e-36, normal)
        assert worst <= eps


def test_results_written_in_place_are_seen_by_autograd():
    """A tensor that a pending backward saved and one of these calls then overwrote is
    reported, as for torch's own operations in place."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.grads import clip_grads, grad_norm
    from mxfp4_routed_expert_gemv_amd.w4 import w4_glu, w4_linear
    x = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    codes = torch.full((64, 32), 0x9A, dtype=torch.uint8, device="cuda")
    scale = torch.ones((64, 2), dtype=torch.bfloat16, device="cuda")
    other = torch.ones((2, 64), device="cuda")
    calls = [("clip", lambda t: clip_grads([other, t], 1e-3)),
             ("clip into", lambda t: clip_grads([other], 1e-3, out=[t])),
             ("clip into, from an iterator", lambda t: clip_grads(iter([other]), 1e-3, out=iter([t]))),
             ("linear", lambda t: w4_linear(x, codes, scale, out=t)),
             ("gated", lambda t: w4_glu(x, codes, scale, out=t))]
    for name, call in calls:
        p = torch.ones((2, 32 if name == "gated" else 64), device="cuda", requires_grad=True)
        saved = p * 1.0
        loss = (saved * saved).sum()
        call(saved.detach())
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
        assert p.grad is None, name
    # what is only read is not
    p = torch.ones(64, device="cuda", requires_grad=True)
    saved = p * 1.0
    loss = (saved * saved).sum()
    grad_norm([saved.detach()])
    clip_grads([saved.detach()], 1e-3, out=[torch.empty_like(other[0])])
    loss.backward()
    assert (p.grad == 2).all()


@pytest.mark.parametrize("xd", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,n,k", [(40, 4096, 7168), (64, 4096, 7168), (100, 2048, 2048), (200, 512, 4096)])
def test_w4_pieces_of_the_contraction_fill_one_round(T, n, k, xd):
    """The contraction is cut so that its workgroups (128 weight rows x 32 tokens of
    fp32 x, 64 of bf16, x the pieces) make one round of the 256 CUs, which the partial
    sums that a call leaves in its workspace show."""
    require_gpu()
    from test_gpu_dense import rounded, w4_bounds, w4_problem, within
    from mxfp4_routed_expert_gemv_amd import k3moe_w4_workspace_bytes, make_w4
    from mxfp4_routed_expert_gemv_amd.w4 import w4_linear
    x, codes, scale, z = w4_problem(T, n, k, 128, True, xd, 200)
    nbytes = k3moe_w4_workspace_bytes(make_w4(n, k, 128, codes, scale, z), T)
    ws = torch.full((nbytes + 1024,), 0xFF, dtype=torch.uint8, device="cuda")
    out = w4_linear(x, codes, scale, z, out_dtype=torch.float32, workspace=ws)
    torch.cuda.synchronize()
    sums = ws[:nbytes].view(torch.float32)
    used = int((~torch.isnan(sums)).sum())
    pieces = used // (T * n)
    log(f"  T={T} n={n} k={k} {xd}: {pieces} pieces")
    assert used == pieces * T * n and not torch.isnan(sums[:used]).any()
    tokens = 32 if xd == torch.float32 else 64
    assert pieces >= 1 and pieces * -(-n // 128) * -(-T // tokens) <= 256
    assert (ws[nbytes:] == 0xFF).all()
    want, tol = w4_bounds(x, codes, scale, z)
    within(out, want, rounded(want, tol, torch.float32), 0, "linear")


def offset_sums(x, codes, scale, zero):
    """x W^T in 64 bits, and the square of what fp32 roundings leave of it, per output.
    The kernels take a step of 32 weights as sum (16 + q) x - (16 + z) sum x, either sum
    by three matrix instructions, one for each 8 bits of x.  An instruction adds 32
    products to what is there, with a rounding each at most: the first has the partial
    sums, the other two move the full one by 2^-8 of it or less, so that each of their
    64 roundings is of the full sum.  Then the difference is rounded, and the running
    sum of the steps.  A rounding to the nearest is off by at most 2^-24 of its value,
    evenly spread a third of that squared on average, and independent roundings add up
    as their squares."""
    n, half = codes.shape
    k, T = 2 * half, x.shape[0]
    q = torch.stack([codes & 15, codes >> 4], -1).view(n, k).to(F8)
    z = (torch.full_like(scale, 8.0) if zero is None else zero).to(F8).repeat_interleave(k // scale.shape[1], 1)
    s = scale.to(F8).repeat_interleave(k // scale.shape[1], 1)
    xs = x.to(F8).view(T, k // 32, 32).transpose(0, 1).contiguous()     # [steps][T][32]
    qs = (16 + q).view(n, k // 32, 32).permute(1, 2, 0).contiguous()    # [steps][32][n]
    zs = (16 + z)[:, ::32].t()[:, None, :]
    dot = off = squares = 0
    for i in range(32):
        dot = dot + xs[:, :, i:i + 1] * qs[:, i:i + 1]
        off = off + xs[:, :, i:i + 1] * zs
        squares = squares + dot ** 2 + off ** 2
    squares = squares + 64 * (dot ** 2 + off ** 2)
    ss = s[:, ::32].t()[:, None, :]
    term = (dot - off) * ss
    run = term.cumsum(0)
    return run[-1], (S24 ** 2 / 3) * (squares * ss ** 2 + term ** 2 + run ** 2).sum(0)


FP32_X = [(1, 96, 1024, 128), (3, 500, 4096, 128), (8, 130, 2048, 256), (13, 66, 1536, 512), (16, 40, 640, 64),
          (30, 200, 1024, 128), (48, 258, 2048, 64), (200, 70, 1024, 128), (5, 514, 4096, 32), (70, 100, 1120, 32)]


@pytest.mark.parametrize("mean", [0.0, 0.5, 20.0])
@pytest.mark.parametrize("T,n,k,group", FP32_X)
def test_w4_fp32_values_keep_fp32s_bits(T, n, k, group, mean):
    """fp32 x into fp32 outputs: the error of all outputs together is that of fp32
    roundings, for x with a mean too (where the offset's sums are far larger than their
    difference), for zero points past 15 and for scales of either sign.  An x without
    its lowest 8 bits is off by more, without its lower 16 by hundreds of times."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.w4 import w4_linear
    g = torch.Generator().manual_seed(300 + T)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8).cuda()
    shape = (n, k // group)
    sign = torch.randint(0, 2, shape, generator=g) * 2 - 1
    scale = ((torch.rand(shape, generator=g) * 0.1 + 0.01) * sign).bfloat16().cuda()
    x = (torch.randn((T, k), generator=g) + mean).cuda()
    for hi in (None, 16, 256):
        zero = None if hi is None else torch.randint(hi // 2, hi, shape, generator=g, dtype=torch.int64).to(torch.uint8).cuda()
        want, square = offset_sums(x, codes, scale, zero)
        got = w4_linear(x, codes, scale, zero, out_dtype=torch.float32)
        torch.cuda.synchronize()
        # (and the waves' and pieces' sums, 64 at most, a rounding of about the output each)
        allowed = float((square + 64 / 3 * (S24 * want) ** 2).sum()) ** 0.5
        err = float((got.to(F8) - want).norm())
        log(f"  T={T} n={n} k={k} group={group} mean={mean} zero<{hi}: {err:.3e} of {allowed:.3e}, "
            f"relative {err / float(want.norm()):.2e}")
        assert err <= allowed


@pytest.mark.parametrize("T,n,k,group", FP32_X[:8])
def test_w4_fp32_values_do_not_depend_on_how_scales_are_grouped(T, n, k, group):
    """A longer group is groups of 32 with one scale: fp32 x into fp32 outputs takes the
    offset off after every 32 weights, before its sums grow, whatever the group, so the
    bits are the same."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.w4 import w4_glu, w4_linear
    from test_gpu_dense import w4_problem
    x, codes, scale, zero = w4_problem(T, n, k, group, True, torch.float32, 320)
    fine = [t.repeat_interleave(group // 32, 1).contiguous() for t in (scale, zero)]
    x += 3.0
    for call in (w4_linear, w4_glu):
        got, want = call(x, codes, scale, zero), call(x, codes, *fine)
        torch.cuda.synchronize()
        assert torch.equal(got, want), call.__name__


@pytest.mark.parametrize("part", [9, 17, 18])
@pytest.mark.parametrize("group", [32, 64, 128, 512])
@pytest.mark.parametrize("T", [1, 2, 7, 16, 25, 33, 70, 260])
def test_w4_low_bits_of_fp32_values(T, group, part):
    """Outputs that the low bits of x alone make up: in every 128 weights one pair of x, 1
    and 1 + 2^-part, meets weights 7 and -7, the rest of x is zero.  31 + 17 (1 + 2^-18)
    has 24 bits, so every sum here is exact in fp32, and the output -7 (k / 128) 2^-part."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.w4 import w4_glu, w4_linear
    n, k = 48, 1536
    codes = torch.full((n, k // 2), 0x1F, dtype=torch.uint8, device="cuda")   # 15, 1, 15, 1, ...
    scale = torch.ones((n, k // group), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((T, k), device="cuda")
    for b in range(k // 128):   # (another place of the block in every block and token)
        for t in range(T):
            at = 128 * b + 2 * ((5 * b + 7 * t) % 64)
            x[t, at], x[t, at + 1] = 1.0, 1.0 + 2.0 ** -part
    want = -7.0 * (k // 128) * 2.0 ** -part
    got = w4_linear(x, codes, scale)
    both = w4_glu(x, codes, scale)
    torch.cuda.synchronize()
    assert got.dtype == torch.float32 and (got == want).all()
    # silu(g) u with g = u = want, small: the sigmoid's and two products' roundings
    h = want * want / (1 + math.exp(-want))
    assert ((both.to(F8) - h).abs() <= 16 * S24 * h).all()


@pytest.mark.parametrize("T", [1, 16, 200])
def test_shared_full_size_layer_with_few_tokens(T, monkeypatch):
    """The sizes whose dx is split over the contraction (of two parts a value up to 16
    tokens) and whose weight gradients run on tiles of their own, or share a launch."""
    import test_gpu_dense as dense
    dense.test_shared_train_and_backward(T, 7168, 2048, 2)
    if T <= 16:
        dense.test_shared_values_of_few_tokens_keep_16_bits(T, 7168, 2048, 2, monkeypatch)


@pytest.mark.parametrize("T", [2500, 4096, 16384])
def test_shared_full_size_layer_with_many_tokens(T):
    """256 x 256 tiles over several rounds, full ones and not, and dx in a launch of its
    own: sampled tokens of y, gu and dx and sampled features of the weights' gradients
    against the formulas."""
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.shared import shared_ffn_backward, shared_ffn_train
    from test_gpu_dense import Ref, normal, problem, rounded, within
    d, fs, S = 7168, 2048, 2
    x, w13, w2 = problem(T, d, fs, S, 400)
    y, gu = shared_ffn_train(x, w13, w2)
    dy = normal((T, d), 405, 0.1)
    dx, dw13, dw2 = shared_ffn_backward(x, gu, dy, w13, w2)
    torch.cuda.synchronize()
    # tokens: of every tile of 256 rows one, at another place in each, and the last
    rows = torch.tensor(sorted({min(256 * i + 37 * i % 256, T - 1) for i in range(-(-T // 256))} | {0, T - 1})).cuda()
    ref = Ref(x[rows], w13, w2)
    y_want, y_tol, gu_want, gu_tol = ref.forward()
    within(y[rows], y_want, rounded(y_want, y_tol), 2, "y")
    within(gu[rows], gu_want, gu_tol, 1, "gu")
    want, tol = ref.backward(gu[rows], dy[rows])[0]
    within(dx[rows], want, rounded(want, tol), 2, "dx")
    # features: one of every 128, and the last
    cols = torch.tensor(sorted({128 * i + 29 * i % 128 for i in range(fs // 128)} | {0, fs - 1})).cuda()
    few, xa, dya = T * S24, x.to(F8).abs(), dy.to(F8).abs()
    for j in range(S):
        g, u, w = gu[:, j, cols].to(F8), gu[:, j, fs + cols].to(F8), w2[j].to(F8)[:, cols]
        s = torch.sigmoid(g)
        dh, dh_e = dy.to(F8) @ w, d * S24 * (dya @ w.abs())
        sil, ds, ds_m = g * s, s * (1 + g * (1 - s)), s + (g * s * (1 - s)).abs()
        for name, at, v, e in (("gate", cols, dh * u * ds, (dh_e * ds.abs() + 16 * S24 * (dh.abs() + dh_e) * ds_m) * u.abs()),
                               ("up", fs + cols, dh * sil, (dh_e + 16 * S24 * (dh.abs() + dh_e)) * sil.abs())):
            e = e + B * (v.abs() + e)   # the rounding of dg or du
            want = v.t() @ x.to(F8)
            tol = e.t() @ xa + few * ((v.abs() + e).t() @ xa)
            within(dw13[j][at], want, rounded(want, tol), 2, f"dw13 ({name}) of expert {j}")
        h = sil * u
        want = dy.to(F8).t() @ h
        h_e = (B + 16 * S24) * h.abs()
        within(dw2[j][:, cols], want, rounded(want, dya.t() @ h_e + few * (dya.t() @ (h.abs() + h_e))), 2,
               f"dw2 of expert {j}")


@pytest.mark.parametrize("on_side", [False, True])
def test_the_calls_of_the_c_interface_from_python(on_side):
    """k3moe_* with buffers of the caller's own, on torch's current stream and on one
    given as an object and as a raw handle, against the torch-facing calls."""
    require_gpu()
    import mxfp4_routed_expert_gemv_amd as k3
    from mxfp4_routed_expert_gemv_amd.grads import clip_grads, grad_norm
    from mxfp4_routed_expert_gemv_amd.w4 import w4_glu, w4_linear
    from test_gpu_dense import w4_problem
    T, n, k, group = 40, 96, 512, 64
    x, codes, scale, z = w4_problem(T, n, k, group, True, torch.bfloat16, 500)
    w = k3.make_w4(n, k, group, codes, scale, z)
    need = k3.k3moe_w4_workspace_bytes(w, T)
    linear, gated = w4_linear(x, codes, scale, z), w4_glu(x, codes, scale, z)
    grads = [linear.float(), gated.float()]
    norm, outs = grad_norm(grads), [torch.empty_like(g) for g in grads]
    clip_grads(grads, 0.5, out=outs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream() if on_side else None
    for stream in (side, side.cuda_stream if on_side else None):
        a, b = torch.full_like(linear, 7), torch.full_like(gated, 7)
        ws = torch.empty(max(need, k3.k3moe_grad_workspace_bytes(2)), dtype=torch.uint8, device="cuda")
        mine, got = [torch.full_like(g, 7) for g in grads], torch.full((2,), 7.0, device="cuda")
        ts = (k3.Tensor * 2)()
        for t, g, o in zip(ts, grads, mine):
            t.data, t.out, t.numel, t.dtype, t.out_dtype = g.data_ptr(), o.data_ptr(), g.numel(), k3.F32, k3.F32
        torch.cuda.synchronize()
        k3.k3moe_w4_linear(w, T, k3.BF16, k3.BF16, x, a, ws, stream)
        k3.k3moe_w4_glu(w, T, k3.BF16, k3.BF16, x, b, (ws.data_ptr(), need), stream)
        k3.k3moe_grad_norm(ts, 2, got[:1], ws, stream)
        k3.k3moe_grad_clip(ts, 2, 0.5, got[1:], ws, stream)
        torch.cuda.synchronize()
        assert torch.equal(a, linear) and torch.equal(b, gated)
        assert torch.equal(got, torch.stack([norm, norm]))
        assert all(torch.equal(p, q) for p, q in zip(mine, outs))
    with pytest.raises(k3.K3moeError, match="workspace"):
        k3.k3moe_w4_linear(w, T, k3.BF16, k3.BF16, x, linear, None, None)
    with pytest.raises(k3.K3moeError, match="overlaps"):
        k3.k3moe_w4_glu(w, T, k3.BF16, k3.BF16, x, x, ws, None)
