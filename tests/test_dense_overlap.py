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
