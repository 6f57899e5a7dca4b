"""Argument checks of the orthogonalised update, on the CPU: every invalid call is
refused with the documented status before anything is launched."""
import ctypes
import math

import pytest
import torch

k3 = pytest.importorskip("mxfp4_routed_expert_gemv_amd")

EINVAL, ESHAPE, EALIGN, EWORKSPACE, EUNSUPPORTED = 1, 2, 3, 4, 5
G, OUT, WS = 0x10000000, 0x20000000, 0x30000000
MUON = (3.4445, -4.7750, 2.0315)


def problem(batch=1, m=64, n=128, dtype=None, steps=5, coefficients=None, scale=1.0):
    flat = list(MUON) * max(steps, 0) if coefficients is None else list(coefficients)
    c = (ctypes.c_float * max(len(flat), 1))(*flat)
    return k3.Ortho(batch, m, n, k3.F32 if dtype is None else dtype, steps, c, scale)


def call(p, g=G, out=OUT, ws=WS, ws_bytes=1 << 27):
    return k3.lib.k3moe_orthogonalize(None if p is None else ctypes.byref(p), g, out, ws, ws_bytes, None)


def test_refusals():
    assert call(None) == EINVAL
    for kw in (dict(batch=0), dict(batch=65536), dict(m=0), dict(n=0), dict(m=-3), dict(m=32769),
               dict(n=32769), dict(batch=65535, m=1024, n=1024)):
        assert call(problem(**kw)) == ESHAPE, kw
    assert call(problem(dtype=2)) == EUNSUPPORTED
    assert call(problem(steps=0)) == EINVAL
    assert call(problem(steps=65)) == EINVAL
    p = problem()
    p.coefficients = None
    assert call(p) == EINVAL
    for s in (math.inf, math.nan):
        assert call(problem(scale=s)) == EINVAL
    assert call(problem(), g=None) == EINVAL
    assert call(problem(), out=None) == EINVAL
    assert call(problem(), g=G + 8) == EALIGN
    assert call(problem(), out=OUT + 2) == EALIGN
    assert call(problem(), ws=None, ws_bytes=0) == EWORKSPACE
    assert call(problem(), ws_bytes=256) == EWORKSPACE
    assert call(problem(), ws=WS + 16) == EALIGN


def test_overlaps():
    p, size = problem(), 64 * 128 * 4
    assert call(p, out=G) == EINVAL                  # fp32: not in place
    assert call(p, out=G + size - 16) == EINVAL
    b = problem(dtype=k3.BF16)
    assert call(b, out=G + 16) == EINVAL             # (in place only as a whole)
    need = k3.k3moe_orthogonalize_workspace_bytes(p)
    assert call(p, ws=G) == EINVAL
    assert call(p, ws=G - need + 256) == EINVAL
    assert call(p, ws=OUT) == EINVAL


@pytest.mark.parametrize("c,ok", [
    (MUON, True), ((1.5, -0.5, 0.0), True), ((1.875, -1.25, 0.375), True), ((1.0, 0.0, 0.0), True),
    ((4.0, 0.0, 0.0), False),             # 1 -> 4
    ((3.4445, -4.7750, 2.5), False),      # 1 -> 1.17 -> 2.0
    ((0.5, 3.5, -3.95), True),            # highest in the middle
    ((0.0, 16.0, -16.0), False),          # |b y + c y^2| = 4 at 1 / 2
    ((-1.5, 0.5, 0.0), True),             # the same with the sign turned
    ((0.0, 5.0, -4.0), False),            # highest inside: 1 -> 1.3 -> 3.8
    ((0.0, 2.0, -1.0), True),             # a step without the linear term
    ((math.nan, 0.0, 0.0), False), ((1.0, math.inf, 0.0), False)])
def test_the_bound_on_singular_values(c, ok):
    """Against a fine scan of the interval that the singular values can fill."""
    p = problem(coefficients=list(c) * 5)
    top, good = 1.0, all(math.isfinite(v) for v in c)
    for _ in range(5 if good else 0):
        v = torch.linspace(0, top, 20001, dtype=torch.float64)
        y = v * v
        good = good and top <= 1.4 and float((c[1] * y + c[2] * y * y).abs().max()) <= 3.9
        top = float((c[0] * v + c[1] * v ** 3 + c[2] * v ** 5).abs().max())
    assert good == ok, "the scan itself"
    assert (k3.k3moe_orthogonalize_workspace_bytes(p) > 0) == ok


def test_workspace():
    n = k3.k3moe_orthogonalize_workspace_bytes
    assert n(problem(m=64, n=128)) >= 3 * 64 * 128 * 2 + 2 * 64 * 64 * 2
    assert n(problem(m=128, n=64)) == n(problem(m=64, n=128))
    assert n(problem(batch=3)) > n(problem())
    assert n(problem(m=0)) == 0
    # one launch that keeps nothing; and the first sizes past it
    assert n(problem(m=256, n=128)) == 0 and n(problem(m=65, n=65)) == 0
    assert n(problem(m=257, n=128)) and n(problem(m=256, n=129)) and n(problem(m=256, n=64))


def test_python_call_refuses_what_is_not_on_a_gpu():
    from mxfp4_routed_expert_gemv_amd.ortho import orthogonalize
    with pytest.raises(ValueError):
        orthogonalize(torch.zeros(4, 4))
    with pytest.raises(TypeError):
        orthogonalize(torch.zeros(4, 4, dtype=torch.float16))
    with pytest.raises(ValueError):
        orthogonalize(torch.zeros(4))
