"""Calls of the dense operators whose outputs or workspace overlap something else the
call reads or writes are refused on the host, before anything is launched."""
import ctypes

import pytest

k3 = pytest.importorskip("mxfp4_routed_expert_gemv_amd")

EINVAL, EWORKSPACE = 1, 4
BASE = 1 << 32   # addresses that are never dereferenced: validation fails first
T, D, FS, S = 40, 256, 128, 2
STEP = 1 << 26


def places(sizes):
    """A place for every operand, far from each other."""
    return {name: BASE + i * STEP for i, name in enumerate(sizes)}


def refused(status, a, b):
    msg = k3.lib.k3moe_last_error().decode()
    assert status == EINVAL and "overlaps" in msg, (a, b, status, msg)


def each_overlap(sizes, written, call, pairs_ok=()):
    """call(places) with every written operand moved onto another's first and last 16
    bytes, and its own last ones onto the other's first."""
    for a in written:
        for b in sizes:
            if a == b or (a, b) in pairs_ok or (b, a) in pairs_ok:
                continue
            # (the workspace starts at whole 256 bytes)
            unit = 256 if a == "workspace" else 16
            for at in (0, (sizes[b] - 1) // unit * unit, -((sizes[a] - 1) // unit * unit)):
                p = places(sizes)
                if b == "workspace" and at < 0:
                    continue   # covered with a and b exchanged
                p[a] = p[b] + at
                refused(call(p), a, b)


def test_training_forward():
    sh = k3.make_shape(T, D, 32, 1, 1, S, FS, k3.BF16, k3.F32)
    need = k3.k3moe_workspace_bytes(sh, k3.OP_SHARED_TRAIN)
    sizes = {"x": T * D * 2, "w13": S * 2 * FS * D * 2, "w2": S * D * FS * 2, "gu": T * S * 2 * FS * 2,
             "y": T * D * 4, "workspace": need}

    def call(p):
        b = k3.make_bank(k3.FMT_BF16, S, D, FS, p["w13"], None, p["w2"], None)
        return k3.lib.k3moe_shared_ffn_train(ctypes.byref(sh), ctypes.byref(b), p["x"], p["gu"], p["y"],
                                             p["workspace"], need, None)
    each_overlap(sizes, ("gu", "y", "workspace"), call)


def test_training_backward():
    sh = k3.make_shape(T, D, 32, 1, 1, S, FS, k3.BF16, k3.BF16)
    need = k3.k3moe_workspace_bytes(sh, k3.OP_SHARED_BACKWARD)
    sizes = {"x": T * D * 2, "gu": T * S * 2 * FS * 2, "dy": T * D * 2, "w13": S * 2 * FS * D * 2,
             "w2": S * D * FS * 2, "dx": T * D * 2, "dw13": S * 2 * FS * D * 2, "dw2": S * D * FS * 2,
             "workspace": need}

    def call(p, only=None):
        b = k3.make_bank(k3.FMT_BF16, S, D, FS, p["w13"], None, p["w2"], None)
        out = [p[o] if only in (None, o) else None for o in ("dx", "dw13", "dw2")]
        return k3.lib.k3moe_shared_ffn_backward(ctypes.byref(sh), ctypes.byref(b), p["x"], p["gu"], p["dy"],
                                                *out, p["workspace"], need, None)
    outs = ("dx", "dw13", "dw2")
    each_overlap(sizes, outs + ("workspace",), call)
    # one output asked for alone: against all that is read
    for o in outs:
        some = {k: v for k, v in sizes.items() if k not in outs or k == o}
        each_overlap(some, (o,), lambda p: call({**places(sizes), **p}, o))


def test_training_backward_of_an_empty_batch():
    sh = k3.make_shape(0, D, 32, 1, 1, S, FS, k3.BF16, k3.BF16)
    sizes = {"w13": S * 2 * FS * D * 2, "w2": S * D * FS * 2, "dw13": S * 2 * FS * D * 2, "dw2": S * D * FS * 2}

    def call(p):
        b = k3.make_bank(k3.FMT_BF16, S, D, FS, p["w13"], None, p["w2"], None)
        return k3.lib.k3moe_shared_ffn_backward(ctypes.byref(sh), ctypes.byref(b), None, None, None, None,
                                                p["dw13"], p["dw2"], None, 0, None)
    each_overlap(sizes, ("dw13", "dw2"), call)


@pytest.mark.parametrize("glu", [False, True])
def test_w4_workspace(glu):
    """Above 16 tokens the workspace holds partial sums that workgroups write while
    others still read the operands."""
    fn = k3.lib.k3moe_w4_glu if glu else k3.lib.k3moe_w4_linear
    n, k, group = 64, 512, 128
    scales = n * (k // group)

    def call(p):
        w = k3.make_w4(n, k, group, p["codes"], p["scale"], p["zero"])
        return fn(ctypes.byref(w), T, k3.F32, k3.BF16, p["x"], p["out"], p["workspace"], need, None)
    need = k3.k3moe_w4_workspace_bytes(k3.make_w4(n, k, group, BASE, BASE, BASE), T)
    assert need > 0
    sizes = {"x": T * k * 4, "codes": n * k // 2, "scale": 2 * scales, "zero": scales,
             "out": T * (n // 2 if glu else n) * 2, "workspace": need}
    each_overlap(sizes, ("out", "workspace"), call)


def grads(*rows):
    ts = (k3.Tensor * len(rows))()
    for t, r in zip(ts, rows):
        t.data, t.out, t.numel, t.dtype, t.out_dtype = r
    return ts


def test_clip_norm_and_workspace():
    """*norm and the partial sums are written while tensors are still read or
    written: neither may lie in a tensor, in an out or in the other."""
    n = 1000
    need = k3.k3moe_grad_workspace_bytes(3)
    sizes = {"data": 2 * n, "out": 4 * n, "second": 4 * n, "norm": 4, "workspace": need}

    def call(p):
        ts = grads((p["data"], p["out"], n, k3.BF16, k3.F32), (p["second"], p["second"], n, k3.F32, k3.F32),
                   (None, None, 0, k3.F32, k3.F32))
        return k3.lib.k3moe_grad_clip(ts, 3, 1.0, p["norm"], p["workspace"], need, None)
    each_overlap(sizes, ("norm", "workspace"), call)
    # the norm's every place inside a tensor
    for at in (0, 4, 2 * n - 4, 4 * n - 4):
        p = places(sizes)
        p["norm"] = p["out"] + at
        refused(call(p), "norm", "out")


def test_norm_and_workspace_of_the_norm_alone():
    """grad_norm writes *norm after everything is read, so it may replace an element;
    its partial sums may not."""
    n = 1000
    need = k3.k3moe_grad_workspace_bytes(1)
    sizes = {"data": 2 * n, "norm": 4, "workspace": need}

    def call(p):
        return k3.lib.k3moe_grad_norm(grads((p["data"], None, n, k3.BF16, 7)), 1, p["norm"], p["workspace"],
                                      need, None)
    each_overlap(sizes, ("workspace",), call)
