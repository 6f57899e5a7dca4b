"""Argument checks of the dense operators (the shared experts' training pass,
4-bit products, gradient norm and clipping) on the CPU: every invalid call is
refused with the documented status before anything is launched."""
import ctypes

import pytest
import torch

k3 = pytest.importorskip("mxfp4_routed_expert_gemv_amd")

EINVAL, ESHAPE, EALIGN, EWORKSPACE, EUNSUPPORTED = 1, 2, 3, 4, 5
FAKE = 0x100000   # an aligned address that is never dereferenced: validation fails first


def shape(T=8, **kw):
    a = dict(T=T, d=256, f=32, E=1, k=1, n_shared=2, f_shared=128, x_dtype=k3.BF16,
             out_dtype=k3.BF16)
    a.update(kw)
    return k3.make_shape(**a)


def bank(n=2, d=256, f=128, w13=FAKE, w2=FAKE, fmt=None):
    return k3.make_bank(k3.FMT_BF16 if fmt is None else fmt, n, d, f, w13, None, w2, None)


def train(s, b, x=FAKE, gu=FAKE, y=FAKE, ws=(FAKE, 1 << 40)):
    return k3.lib.k3moe_shared_ffn_train(ctypes.byref(s), ctypes.byref(b), x, gu, y, ws[0], ws[1],
                                         None)


def backward(s, b, x=FAKE, gu=FAKE, dy=FAKE, dx=FAKE, dw13=FAKE, dw2=FAKE, ws=(FAKE, 1 << 40)):
    return k3.lib.k3moe_shared_ffn_backward(ctypes.byref(s), ctypes.byref(b), x, gu, dy, dx, dw13,
                                            dw2, ws[0], ws[1], None)


@pytest.mark.parametrize("call", [train, backward])
def test_shared_training_refusals(call):
    assert call(shape(), bank(fmt=k3.FMT_MXFP4)) == EUNSUPPORTED
    assert call(shape(x_dtype=k3.F32), bank()) == EUNSUPPORTED
    assert call(shape(n_shared=0), bank(n=0)) == EINVAL
    assert call(shape(), bank(n=3)) == EINVAL
    assert call(shape(), bank(f=64)) == EINVAL
    assert call(shape(d=250), bank(d=250)) == ESHAPE
    assert call(shape(T=-1), bank()) == EINVAL
    assert call(shape(T=(1 << 26) + 1), bank()) == ESHAPE
    assert call(shape(), bank(w13=None)) == EINVAL
    assert call(shape(), bank(w2=FAKE + 8)) == EALIGN
    assert call(shape(), bank(), x=None) == EINVAL
    assert call(shape(), bank(), gu=FAKE + 2) == EALIGN
    assert call(shape(), bank(), ws=(None, 0)) == EWORKSPACE
    assert call(shape(), bank(), ws=(FAKE, 256)) == EWORKSPACE
    assert call(shape(), bank(), ws=(FAKE + 16, 1 << 40)) == EALIGN


def test_shared_training_outputs_and_empty_batch():
    assert train(shape(), bank(), y=None) == EINVAL
    assert train(shape(T=0), bank(), x=None, gu=None, y=None, ws=(None, 0)) == 0
    assert backward(shape(), bank(), dy=None) == EINVAL
    assert backward(shape(), bank(), dx=FAKE + 4) == EALIGN
    assert backward(shape(), bank(), dw2=FAKE + 4) == EALIGN
    # no gradient asked for: nothing to do
    assert backward(shape(), bank(), dx=None, dw13=None, dw2=None) == 0
    assert backward(shape(T=0), bank(), x=None, gu=None, dy=None, dx=None, dw13=None, dw2=None,
                    ws=(None, 0)) == 0


def test_shared_training_workspace():
    assert k3.k3moe_workspace_bytes(shape(), k3.OP_SHARED_TRAIN) >= 8 * 256 * 2
    assert k3.k3moe_workspace_bytes(shape(), k3.OP_SHARED_BACKWARD) >= 3 * 8 * 256 * 2
    assert k3.k3moe_workspace_bytes(shape(T=0), k3.OP_SHARED_BACKWARD) == 0
    assert k3.k3moe_workspace_bytes(shape(d=100), k3.OP_SHARED_TRAIN) == 0


def w4(n=64, k=256, group=128, codes=FAKE, scale=FAKE, zero=None):
    return k3.make_w4(n, k, group, codes, scale, zero)


@pytest.mark.parametrize("glu", [False, True])
def test_w4_refusals(glu):
    fn = k3.lib.k3moe_w4_glu if glu else k3.lib.k3moe_w4_linear

    def call(w, T=1, xd=k3.BF16, od=k3.BF16, x=FAKE, out=FAKE, ws=(None, 0)):
        return fn(ctypes.byref(w), T, xd, od, x, out, ws[0], ws[1], None)
    assert fn(None, 1, k3.BF16, k3.BF16, FAKE, FAKE, None, 0, None) == EINVAL
    assert call(w4(), T=-1) == EINVAL
    assert call(w4(n=-2)) == EINVAL
    assert call(w4(n=0)) == ESHAPE
    assert call(w4(n=(1 << 20) + 2)) == ESHAPE
    assert call(w4(k=0)) == ESHAPE
    assert call(w4(k=200)) == ESHAPE
    assert call(w4(k=(1 << 20) + 128)) == ESHAPE
    assert call(w4(n=1 << 20, k=1 << 17)) == ESHAPE   # 2^37 weights
    for g in (0, 16, 48, 96, 192):
        assert call(w4(k=g * 4 or 64, group=g)) == ESHAPE, g
    assert call(w4(group=512)) == ESHAPE          # longer than a row
    assert call(w4(), T=(1 << 18) + 1) == ESHAPE
    assert call(w4(), xd=2) == EUNSUPPORTED
    assert call(w4(), od=7) == EUNSUPPORTED
    assert call(w4(codes=None)) == EINVAL
    assert call(w4(scale=FAKE + 2)) == EALIGN
    assert call(w4(zero=FAKE + 1)) == EALIGN
    assert call(w4(), x=None) == EINVAL
    assert call(w4(), out=FAKE + 8) == EALIGN
    assert call(w4(codes=None), T=0, x=None, out=None) == 0
    if glu:
        assert call(w4(n=63)) == ESHAPE
    # the workspace: none up to 16 tokens, then partial sums
    assert k3.k3moe_w4_workspace_bytes(w4(), 16) == 0
    assert k3.k3moe_w4_workspace_bytes(w4(n=0), 17) == 0
    need = k3.k3moe_w4_workspace_bytes(w4(), 17)
    assert need >= 17 * 64 * 4 and need % 256 == 0
    assert k3.k3moe_w4_workspace_bytes(w4(n=7168, k=7168), 1 << 18) <= 1 << 28
    assert call(w4(), T=17) == EWORKSPACE
    assert call(w4(), T=17, ws=(FAKE, need - 256)) == EWORKSPACE
    assert call(w4(), T=17, ws=(FAKE + 16, need)) == EALIGN


def tensors(*rows):
    ts = (k3.Tensor * len(rows))()
    for t, r in zip(ts, rows):
        t.data, t.out, t.numel, t.dtype, t.out_dtype = r
    return ts


ROW = (FAKE, FAKE, 100, k3.F32, k3.F32)


@pytest.mark.parametrize("clip", [False, True])
def test_gradient_refusals(clip):
    def call(ts, n=None, norm=FAKE, ws=(FAKE, 1 << 30)):
        n = len(ts) if n is None else n
        if clip:
            return k3.lib.k3moe_grad_clip(ts, n, 1.0, norm, ws[0], ws[1], None)
        return k3.lib.k3moe_grad_norm(ts, n, norm, ws[0], ws[1], None)
    ok = tensors(ROW)
    assert call(ok, n=-1) == EINVAL
    assert call(ok, n=(1 << 20) + 1) == EINVAL
    assert call(None, n=1) == EINVAL
    assert call(ok, norm=None) == EINVAL
    assert call(ok, norm=FAKE + 2) == EALIGN
    assert call(ok, ws=(None, 0)) == EWORKSPACE
    assert call(ok, ws=(FAKE, 64)) == EWORKSPACE
    assert call(ok, ws=(FAKE + 8, 1 << 30)) == EALIGN
    assert call(tensors((FAKE, FAKE, -1, 0, 0))) == EINVAL
    assert call(tensors((FAKE, FAKE, (1 << 40) + 1, 0, 0))) == EINVAL
    assert call(tensors((None, FAKE, 4, 0, 0))) == EINVAL
    assert call(tensors((FAKE, FAKE, 4, 2, 0))) == EUNSUPPORTED
    assert call(tensors((FAKE + 2, FAKE, 4, k3.F32, 0))) == EALIGN
    assert call(tensors((FAKE + 1, FAKE, 4, k3.BF16, 1))) == EALIGN


def test_clip_refusals():
    def call(ts, max_norm=1.0):
        # no workspace: a list that passes every other check ends there
        return k3.lib.k3moe_grad_clip(ts, len(ts), max_norm, FAKE, None, 0, None)
    assert call(tensors(ROW), -1.0) == EINVAL
    assert call(tensors(ROW), float("nan")) == EINVAL
    assert call(tensors(ROW), float("inf")) == EWORKSPACE
    assert call(tensors((FAKE, None, 4, 0, 0))) == EINVAL
    assert call(tensors((FAKE, FAKE, 4, 0, 2))) == EUNSUPPORTED
    assert call(tensors((FAKE, FAKE + 2, 4, 0, k3.F32))) == EALIGN
    far = FAKE + (1 << 20)
    # in place, and into buffers of their own
    assert call(tensors(ROW, (far, far + 4096, 100, k3.BF16, k3.F32))) == EWORKSPACE
    # neighbours that touch do not overlap
    assert call(tensors((FAKE, FAKE, 100, 0, 0), (FAKE + 400, FAKE + 400, 4, 0, 0))) == EWORKSPACE
    # the same tensor twice, in place; two outputs in one place; an output over
    # another tensor's data; over a part of its own; its own in another type
    assert call(tensors(ROW, ROW)) == EINVAL
    assert call(tensors((FAKE, far, 100, 0, 0), (FAKE + 400, far + 396, 100, 0, 0))) == EINVAL
    assert call(tensors((FAKE, far, 100, 0, 0), (far + 100, far + 4096, 4, 0, 0))) == EINVAL
    assert call(tensors((FAKE, FAKE + 4, 100, 0, 0))) == EINVAL
    assert call(tensors((FAKE, FAKE, 100, k3.F32, k3.BF16))) == EINVAL
    # a wide span before and a small one inside it, not next to each other in order
    assert call(tensors((FAKE, FAKE, 1000, 0, 0), (FAKE + 4000, FAKE + 4000, 4, 0, 0),
                        (FAKE + 400, far, 4, 0, 0))) == EINVAL
    # reading the same data into two outputs is fine; empty tensors have no place
    assert call(tensors((FAKE, far, 100, 0, 0), (FAKE, far + 400, 100, 0, 0))) == EWORKSPACE
    assert call(tensors(ROW, (None, None, 0, 0, 0))) == EWORKSPACE


def test_gradient_workspace_grows_with_the_list():
    sizes = [k3.k3moe_grad_workspace_bytes(n) for n in (0, 1, 12, 400, 1 << 20)]
    assert sizes == sorted(sizes) and all(s % 256 == 0 and s > 0 for s in sizes)
    assert k3.k3moe_grad_workspace_bytes(-1) == 0
    assert k3.k3moe_grad_workspace_bytes((1 << 20) + 1) == 0


def test_python_checks():
    from mxfp4_routed_expert_gemv_amd import grads, shared, w4 as w4mod
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w13, w2 = (torch.zeros(s, dtype=torch.bfloat16) for s in ((1, 256, 256), (1, 256, 128)))
    with pytest.raises(TypeError):
        shared.shared_ffn_train(x.float(), w13, w2)
    with pytest.raises(ValueError):
        shared.shared_ffn_train(x[:, :128], w13, w2)
    with pytest.raises(ValueError):
        shared.shared_ffn_train(x.t().contiguous().t(), w13, w2)
    with pytest.raises(ValueError):
        shared.shared_ffn_backward(x, torch.zeros(4, 1, 128, dtype=torch.bfloat16), x, w13, w2)
    codes, scale = torch.zeros(8, 128, dtype=torch.uint8), torch.ones(8, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w4mod.w4_linear(x[:, :128], codes, scale)
    with pytest.raises(TypeError):
        w4mod.w4_linear(x.half(), codes, scale)
    with pytest.raises(TypeError):
        w4mod.w4_linear(x, codes, scale, zero=scale)
    with pytest.raises(TypeError):
        w4mod.w4_linear(x, codes, scale, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        grads.grad_norm([])
    with pytest.raises(TypeError):
        grads.grad_norm([x.half()])
    with pytest.raises(ValueError):
        grads.grad_norm([x.t()])
    with pytest.raises(ValueError):
        grads.clip_grads([x], 1.0, out=[x, x])
    with pytest.raises(ValueError):
        grads.clip_grads([x], 1.0, out=[x[:2]])


def test_a_stream_of_another_device_is_refused():
    import types
    from mxfp4_routed_expert_gemv_amd import on_device
    with pytest.raises(ValueError, match="stream of GPU 1"):
        on_device(torch.device("cuda", 0), types.SimpleNamespace(device_index=1))


@pytest.mark.parametrize("glu", [False, True])
def test_w4_out_must_not_overlap_what_is_read(glu):
    fn = k3.lib.k3moe_w4_glu if glu else k3.lib.k3moe_w4_linear
    far = [FAKE + (i << 24) for i in range(5)]
    T, n, k = 4, 64, 256

    def call(x, codes, scale, zero, out, out_dtype):
        w = k3.make_w4(n, k, 128, codes, scale, zero)
        return fn(ctypes.byref(w), T, k3.BF16, out_dtype, x, out, None, 0, None)
    for od, size in ((k3.BF16, 2), (k3.F32, 4)):
        bytes_out = T * (n // 2 if glu else n) * size
        for i, extent in enumerate((T * k * 2, n * k // 2, n * 2 * 2, n * 2)):
            for at in (far[i], far[i] + extent - 16, far[i] - bytes_out + 16):
                assert call(*far[:4], at, od) == EINVAL, (i, at)
                assert b"overlaps" in k3.lib.k3moe_last_error()


def test_a_workspace_kernels_cannot_use_is_refused():
    from mxfp4_routed_expert_gemv_amd import check_workspace
    with pytest.raises(ValueError, match="workspace"):
        check_workspace(torch.zeros(256, dtype=torch.uint8), 0)   # host memory
