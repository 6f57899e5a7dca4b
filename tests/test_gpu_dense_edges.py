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
