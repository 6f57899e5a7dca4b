"""The orthogonalised update on the GPU against its definition in 64 bits.

Tolerances.  The library's header names what is rounded: the products' operands to
fp16 (X, A = X X^T and B = b A + c A A, each scaled by a power of two), a X to two
fp16 parts (to one in the last step), the result to bf16.  `rounded` takes exactly these roundings in 64 bits,
so its distance E from the definition is what they cost on this input; the kernels
add fp32 sums (2^-24 a term) that move some of them by one step.  The result may be
1.25 E away in norm, and each value by its bf16 rounding, 2^-8 of it, and 8 times
the rms of E (a sum of thousands of independent roundings; of a few values E can be
small by chance, so at least 3 fp16 roundings, 3 x 2^-11 of the rms value, count).
That rms is not the same in every column of X taken wide: a step takes column x to
(a + B) x, with the roundings of B, which all columns share, and those of x's own
values, so what a step adds to a column's error is proportional to the column's norm.
The norm starts at the gradient's column's and ends at the result's: where the larger
of the two is over the mean, the column's bound is so many times larger."""
import pytest
import torch

from gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu

F8 = torch.float64
MUON = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)
QUINTIC = (1.875, -1.25, 0.375)


def call(*a, **kw):
    require_gpu()
    from mxfp4_routed_expert_gemv_amd.ortho import orthogonalize
    return orthogonalize(*a, **kw)


def gradient(batch, m, n, dtype, seed, rank=4, noise=0.05):
    """Some directions over the noise, each half as strong as the one before."""
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.empty(shape, device="cuda").normal_(generator=g)
    r = min(rank, m, n)
    u, v = normal(batch, m, r), normal(batch, r, n)
    t = sum(0.5 ** i * u[:, :, i, None] * v[:, i, None, :] for i in range(r))
    return ((noise * normal(batch, m, n) + 0.25 * t) * 0.01).to(dtype)


def schedule(steps, coefficients):
    return [coefficients] * steps if not isinstance(coefficients[0], tuple) else coefficients


def exact(g, steps=5, coefficients=MUON, scale=1.0):
    outs = []
    for x in g.to(F8):
        norm = torch.linalg.vector_norm(x)
        x = x / norm if float(norm) else x
        wide = x.shape[0] <= x.shape[1]
        x = x if wide else x.t().contiguous()
        for a, b, c in schedule(steps, coefficients):
            A = x @ x.t()
            x = a * x + (b * A + c * A @ A) @ x
        outs.append(scale * (x if wide else x.t()))
    return torch.stack(outs)


def rounded(g, steps=5, coefficients=MUON, scale=1.0):
    """The definition with the stated roundings, but for the last to bf16."""
    def part(x, s):
        return (x * s).to(torch.float16).to(F8) / s
    S = 2.0 ** 15
    outs = []
    for x in g.to(F8):
        norm = torch.linalg.vector_norm(x)
        x = x / norm if float(norm) else x
        wide = x.shape[0] <= x.shape[1]
        x = x if wide else x.t().contiguous()
        for i, (a, b, c) in enumerate(schedule(steps, coefficients)):
            hi = part(x, S)
            x = hi + (part(x - hi, S) if i + 1 < steps else 0.0)
            A = part(hi @ hi.t(), S)
            B = part(b * A + c * A @ A, S / 2)
            x = a * x + B @ hi
        outs.append(scale * (x if wide else x.t()))
    return torch.stack(outs)


def column_factor(g, w):
    along = 0 if g.shape[0] <= g.shape[1] else 1   # the columns of X taken wide

    def factor(x):
        n = x.norm(dim=along, keepdim=True)
        return n / n.square().mean().sqrt().clamp(min=1e-300)
    return torch.maximum(factor(g), factor(w)).clamp(min=1.0)


def check(got, g, name, **kw):
    want, model = exact(g, **kw), rounded(g, **kw)
    assert got.dtype == torch.bfloat16 and got.shape == g.shape
    got = got.to(F8)
    assert torch.isfinite(got).all(), name
    for b in range(g.shape[0]):
        w, err = want[b], (got[b] - want[b]).abs()
        size = float(w.square().mean().sqrt())
        cost = float((model[b].to(torch.bfloat16).to(F8) - w).norm())
        rms = float((model[b] - w).square().mean().sqrt())
        rms = max(rms, 3 * 2.0 ** -11 * size)
        tol = 2.0 ** -8 * w.abs() + 8 * rms * column_factor(g[b].to(F8), w)
        worst = float((err / tol.clamp(min=1e-300)).max())
        floor = 3 * 2.0 ** -11 * size * w.numel() ** 0.5
        rel = float(err.norm()) / max(1.25 * cost, floor, 1e-300)
        if b == 0:
            n = max(float(w.norm()), 1e-300)
            log(f"  {name}: norm of the error {float(err.norm()) / n:.2e} ({rel:.2f} of its bound), worst value {worst:.2f}")
        assert rel <= 1.0 and worst <= 1.0, (name, b, rel, worst)


# batch, m, n: the least; a vector; odd sizes both ways; whole tiles of every size and
# what does not fill them; stacks
SIZES = [(1, 1, 1), (1, 1, 5), (1, 9, 1), (1, 7, 3), (5, 33, 47), (3, 64, 64), (1, 65, 130), (2, 130, 65),
         (1, 256, 128), (1, 16, 256), (1, 200, 1000), (1, 1000, 201), (2, 513, 515), (1, 896, 7168),
         (1, 1024, 1536), (3, 700, 340), (40, 100, 90), (3, 128, 256), (2, 255, 67), (1, 65, 65), (2, 77, 250),
         (1, 2200, 1900), (2, 64, 20000), (1, 20000, 70)]


@pytest.mark.parametrize("batch,m,n", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_against_the_definition(batch, m, n, dtype):
    g = gradient(batch, m, n, dtype, 1)
    check(call(g), g, f"{batch} x {m} x {n}")


# (of six of these steps the squares of the first coefficients grow past 2^15: the
# tiled products take matrices of every size then)
@pytest.mark.parametrize("batch,m,n", [s for s in SIZES if min(s[1:]) <= 128])
def test_small_matrices_on_the_tiled_products(batch, m, n):
    g = gradient(batch, m, n, torch.float32, 1)
    check(call(g, steps=6), g, f"{batch} x {m} x {n}", steps=6)


# (a short side of 65 .. 128 beside a long one up to 256 takes the products' 11 bits)
@pytest.mark.parametrize("batch,m,n", [s for s in SIZES if min(s[1:]) <= 64 or min(s[1:]) <= 128 and max(s[1:]) > 256] + [
    (2, 64, 64), (2, 128, 4099), (3, 61, 33), (1, 65, 32768), (1, 9000, 5), (2, 257, 65), (1, 128, 257)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_small_matrices_keep_more_bits(batch, m, n, dtype):
    """Short sides up to 128: every operand has 22 bits.  What rounding A = X X^T costs
    is at most 2^-22 of its largest eigenvalue, 1, times what five steps multiply a
    small one by, 3.4445^8 = 19800, so 5e-3 of an eigenvalue in the directions where
    the gradient has least, and those are a small part of it: in norm a tenth of that,
    beside the rounding to bf16 of every value."""
    g = gradient(batch, m, n, dtype, 14)
    want = exact(g)
    err = (call(g).to(F8) - want).abs()
    half = torch.ldexp(torch.ones_like(want), torch.frexp(want).exponent - 9)   # half a step of bf16
    rest = (err - half).clamp(min=0.0)
    rel = float((rest.flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)).max())
    log(f"  {batch} x {m} x {n}: {rel:.1e} beside the rounding")
    assert rel <= 5e-4


def test_pieces_of_different_size():
    """Columns of zeros, of tiny and of large values in different pieces of one matrix."""
    g = gradient(2, 40, 3000, torch.float32, 15)
    g[:, :, :700] = 0
    g[:, :, 900:1500] *= 2.0 ** -40
    g[0, :, 1500:] *= 2.0 ** -70
    check(call(g), g, "pieces")
    t = g.transpose(1, 2).contiguous()
    check(call(t), t, "pieces of rows")


def test_largest_tiles():
    """More than a round of 256 x 256 tiles in every product, rows and columns that do
    not fill the last ones, a tall matrix."""
    g = gradient(2, 4200, 4136, torch.bfloat16, 2, rank=16)
    check(call(g), g, "2 x 4200 x 4136")


@pytest.mark.parametrize("noise", [0.005, 0.0005])
def test_few_strong_directions(noise):
    """Ten and a hundred times weaker noise: what the small singular values are after
    five steps depends on every bit of X."""
    g = gradient(1, 512, 1024, torch.float32, 3, rank=16, noise=noise)
    check(call(g), g, f"noise {noise}")


@pytest.mark.parametrize("m,n", [(150, 260), (33, 90), (120, 77)])
@pytest.mark.parametrize("steps,coefficients", [(1, MUON), (2, CUBIC), (12, CUBIC), (8, QUINTIC),
                                                (3, (MUON, QUINTIC, CUBIC))])
def test_steps_and_coefficients(steps, coefficients, m, n):
    g = gradient(2, m, n, torch.float32, 4)
    check(call(g, steps=steps, coefficients=coefficients, scale=0.2), g, f"{steps} steps",
          steps=steps, coefficients=coefficients, scale=0.2)


def test_singular_vectors_and_values():
    """u p(p(.. (v))) v^T from the singular value decomposition in 64 bits."""
    g = gradient(1, 96, 160, torch.float32, 5)
    u, v, vt = torch.linalg.svd(g[0].to(F8), full_matrices=False)
    v = v / v.norm()
    for _ in range(5):
        v = MUON[0] * v + MUON[1] * v ** 3 + MUON[2] * v ** 5
    want = u @ torch.diag(v) @ vt
    assert float((want - exact(g)[0]).norm() / want.norm()) < 1e-9
    got = call(g)[0].to(F8)
    assert float((torch.linalg.svdvals(got) - v.sort(descending=True).values).abs().max()) < 0.02


def test_scale_of_the_gradient():
    """The result does not depend on the gradient's size, whatever the type holds; a
    matrix of zeros stays zero, also in a stack."""
    g = gradient(1, 70, 90, torch.float32, 6)
    want = call(g)
    for p in (-90, -60, 60, 100):   # (the products stay normal numbers: scaled, no bit is lost)
        s = 2.0 ** p
        assert torch.equal(g * s / s, g)
        assert torch.equal(call(g * s), want), p
    z = torch.cat([torch.zeros_like(g), g, torch.zeros_like(g)])
    out = call(z)
    assert not out[0].any() and not out[2].any() and torch.equal(out[1:2], want)
    assert not call(torch.zeros(300, 200, device="cuda", dtype=torch.bfloat16)).any()


def test_zero_rows_and_columns():
    g = gradient(1, 120, 300, torch.float32, 7)
    g[:, 10:40] = 0
    g[:, :, ::3] = 0
    out = call(g)
    check(out, g, "zero rows")
    assert not out[:, 10:40].any() and not out[:, :, ::3].any()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_non_finite_gradients_show(bad):
    g = gradient(2, 100, 140, torch.float32, 8)
    g[0, 3, 5] = bad
    out = call(g)
    assert torch.isnan(out[0]).all()
    assert torch.isfinite(out[1]).all()


def test_shapes_in_place_and_given_outputs():
    g = gradient(6, 48, 80, torch.bfloat16, 9)
    want = call(g)
    assert torch.equal(call(g[2]), want[2])
    assert torch.equal(call(g.view(2, 3, 48, 80)), want.view(2, 3, 48, 80))
    out = torch.empty_like(g)
    v = out._version
    assert call(g, out=out) is out and torch.equal(out, want) and out._version > v
    h = g.clone()
    assert torch.equal(call(h, out=h), want)
    assert call(g[:0]).shape == (0, 48, 80)
    assert call(torch.empty(4, 0, 8, device="cuda")).shape == (4, 0, 8)


def test_refusals():
    require_gpu()
    from mxfp4_routed_expert_gemv_amd import K3moeError
    g = gradient(1, 48, 80, torch.float32, 10)
    for bad, err in ((lambda: call(g.half()), TypeError), (lambda: call(g[0, 0]), ValueError),
                     (lambda: call(g[:, ::2]), ValueError), (lambda: call(g.cpu()), ValueError),
                     (lambda: call(g, out=torch.empty_like(g)), TypeError),
                     (lambda: call(g, out=torch.empty(1, 48, 79, dtype=torch.bfloat16, device="cuda")), ValueError),
                     (lambda: call(g, steps=0), K3moeError), (lambda: call(g, steps=65), K3moeError),
                     (lambda: call(g, coefficients=(1.0, 2.0)), ValueError),
                     (lambda: call(g, coefficients=(4.0, 0.0, 0.0)), K3moeError),
                     (lambda: call(g, coefficients=(float("nan"), 0.0, 0.0)), K3moeError),
                     (lambda: call(g, scale=float("inf")), K3moeError),
                     (lambda: call(g, workspace=torch.empty(512, dtype=torch.uint8, device="cuda")), K3moeError)):
        with pytest.raises(err):
            bad()


def test_another_stream():
    g = gradient(1, 300, 500, torch.bfloat16, 11)
    want = call(g)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = call(g, stream=st)
    st.synchronize()
    assert torch.equal(got, want)


def test_captured_and_replayed():
    """Replays on new gradients, with the program's own work between; two graphs in
    turn that share a workspace."""
    g, h = gradient(1, 300, 500, torch.bfloat16, 12), gradient(2, 80, 60, torch.float32, 13)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call(g, workspace=ws), call(h, workspace=ws)
    torch.cuda.current_stream().wait_stream(st)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph, t in zip(graphs, (g, h)):
        with torch.cuda.graph(graph):
            outs.append(call(t, workspace=ws))
    for i in range(4):
        g.copy_(gradient(1, 300, 500, torch.bfloat16, 20 + i))
        h.copy_(gradient(2, 80, 60, torch.float32, 30 + i))
        graphs[i & 1].replay()
        graphs[~i & 1].replay()
        got = [o.clone() for o in outs]
        assert torch.equal(got[0], call(g)) and torch.equal(got[1], call(h)), i
