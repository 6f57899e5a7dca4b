"""Workloads of the library's dense operators: the shared experts' training
forward and backward (shared.py), products with 4-bit weights and group scales
(w4.py) and the global gradient norm with clipping (grads.py).

A case is a dict of plain values.  `run` computes one pass in plain torch
operations, or, where `own` is true, through the library's entry points;
`exact` computes the same outputs in 64 bits from the definitions.

  train      y, gu = shared_ffn_train(x, w13, w2): S always-on gated experts,
             gu the pre-activations kept for the backward
  backward   dx, dw13, dw2 = shared_ffn_backward(x, gu, dy, w13, w2)
  w4_linear  out = x W^T, W = (code - zero) * scale, one scale per group of
             weights along a row
  w4_glu     silu(x Wg^T) * (x Wu^T), Wg and Wu the two halves of W's rows
  norm       the 2-norm over all gradients of a step
  clip       the gradients scaled to at most max_norm, in the optimizer's type
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SHARED_SIGMA = 0.02   # standard deviation of the shared experts' weights


# ------------------------------------------------------------------ the cases
def _shared(op, name, T, d, fs, S):
    return {"name": name, "op": op, "T": T, "d": d, "fs": fs, "S": S}


def _w4(op, name, T, n, k, group, zero, x, out):
    return {"name": name, "op": op, "T": T, "n": n, "k": k, "group": group, "zero": zero,
            "x": x, "out": out}


def _grads(op, name, count, lo, hi, bf16, out, odd, threshold):
    return {"name": name, "op": op, "count": count, "lo": lo, "hi": hi, "bf16": bf16, "out": out,
            "odd": odd, "threshold": threshold}


def listed():
    return [
        # a handful of tokens through a toy layer: a unit test's or a sweep's step, all latency
        _shared("train", "train, toy layer", 4, 256, 128, 1),
        # one packed sequence of ragged length through the full-size layer
        _shared("train", "train, 1000 tokens", 1000, 7168, 2048, 2),
        # an ordinary micro-batch of fine-tuning
        _shared("train", "train, 4096 tokens", 4096, 7168, 2048, 2),
        # a short ragged batch: the weight gradients weigh more than the tokens
        _shared("backward", "backward, 517 tokens", 517, 7168, 2048, 2),
        # the ordinary micro-batch
        _shared("backward", "backward, 4096 tokens", 4096, 7168, 2048, 2),
        # the largest batch the layer is measured on
        _shared("backward", "backward, 16384 tokens", 16384, 7168, 2048, 2),
        # one token's down projection while generating
        _w4("w4_linear", "4-bit linear, 1 token", 1, 7168, 4096, 128, False, "bf16", "bf16"),
        # a decode batch, asymmetric codes, one of the fine-grained group sizes
        _w4("w4_linear", "4-bit linear, 64 tokens", 64, 7168, 4096, 32, True, "bf16", "bf16"),
        # one token's gated block while generating, both shared experts side by side
        _w4("w4_glu", "4-bit gated, 1 token", 1, 8192, 7168, 128, True, "bf16", "bf16"),
        # drafted tokens checked together, fp32 hidden state, an odd width
        _w4("w4_glu", "4-bit gated, 5 tokens fp32", 5, 4098, 7168, 64, False, "f32", "f32"),
        # the norm over a small model's step: many small tensors, views into one flat buffer
        _grads("norm", "norm, 200 tensors", 200, 64, 400_000, True, "bf16", True, 1.0),
        # clipping the shared experts' and routers' gradients of four layers into fp32
        _grads("clip", "clip, 12 tensors", 12, 6_422_528, 58_720_256, True, "f32", False, 1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["train", "backward", "w4_linear", "w4_glu", "norm", "clip"])
    if op in ("train", "backward"):
        d = 32 * _log(rng, 8, 224)
        fs = 32 * _log(rng, 4, 64)
        S = rng.choice([1, 1, 2, 3])
        most = 16384 * 7168 * 4096 // (d * fs * S)
        c = _shared(op, "", _log(rng, 1, min(16384, most)), d, fs, S)
    elif op in ("w4_linear", "w4_glu"):
        group = rng.choice([32, 64, 128])
        n = _log(rng, 17, 16384)
        c = _w4(op, "", _log(rng, 1, 64), n + n % 2, group * max(1, _log(rng, 128, 16384) // group),
                group, rng.random() < 0.5, rng.choice(["bf16", "bf16", "f32"]),
                rng.choice(["bf16", "f32"]))
    else:
        hi = _log(rng, 1000, 16_000_000)
        count = min(_log(rng, 1, 400), 1 + 300_000_000 // hi)
        c = _grads(op, "", min(count, 60) if op == "clip" else count, max(1, hi // rng.choice([1, 10, 1000])),
                   hi, rng.random() < 0.7, rng.choice(["bf16", "f32"]), rng.random() < 0.5,
                   rng.choice([0.5, 1.0, 2.0]))
    del c["name"]
    return c


def _sizes(case):
    """The tensors' element counts: spread over lo .. hi by their logarithm, no two orders alike."""
    n, lo, hi = case["count"], case["lo"], case["hi"]
    if n == 1:
        return [hi]
    place = [(7 * i) % n if n % 7 else i for i in range(n)]
    return [int(round(lo * (hi / lo) ** (p / (n - 1)))) for p in place]


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g)
        return t if dtype == torch.float32 else t.to(dtype)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.uint8)

    s = {"case": case}
    if case["op"] in ("train", "backward"):
        T, d, fs, S = (case[k] for k in ("T", "d", "fs", "S"))
        s["x"] = normal(T, d)
        s["w13"] = normal(S, 2 * fs, d, std=SHARED_SIGMA)
        s["w2"] = normal(S, d, fs, std=SHARED_SIGMA)
        if case["op"] == "backward":
            # pre-activations with the spread that x and w13 give
            s["gu"] = normal(T, S, 2 * fs, std=SHARED_SIGMA * math.sqrt(d))
            s["dy"] = normal(T, d, std=0.01)
    elif case["op"] in ("w4_linear", "w4_glu"):
        T, n, k, group = (case[v] for v in ("T", "n", "k", "group"))
        s["x"] = normal(T, k, dtype=DT[case["x"]])
        s["codes"] = whole(0, 256, n, k // 2)
        s["scale"] = (torch.rand((n, k // group), generator=g, device="cuda") * 0.008 + 0.002).bfloat16()
        s["zero"] = whole(5, 11, n, k // group) if case["zero"] else None
    else:
        sizes = _sizes(case)
        src = torch.bfloat16 if case["bf16"] else torch.float32
        odd = int(case["odd"])
        flat = normal(sum(sizes) + odd * len(sizes), std=0.001, dtype=src)
        at = [sum(sizes[:i]) + odd * i for i in range(len(sizes))]
        s["grads"] = [flat[a + odd: a + odd + n] for a, n in zip(at, sizes)]
        if case["op"] == "clip":
            s["outs"] = [torch.empty(n, dtype=DT[case["out"]], device="cuda") for n in sizes]
            # the threshold against the norm these gradients have: half of it, at it or over it
            s["max_norm"] = case["threshold"] * 0.0007 * math.sqrt(sum(sizes))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    op, case = s["case"]["op"], s["case"]
    if op in ("train", "backward"):
        from mxfp4_routed_expert_gemv_amd.shared import shared_ffn_backward, shared_ffn_train
        if op == "train":
            return shared_ffn_train(s["x"], s["w13"], s["w2"])
        return shared_ffn_backward(s["x"], s["gu"], s["dy"], s["w13"], s["w2"])
    if op in ("w4_linear", "w4_glu"):
        from mxfp4_routed_expert_gemv_amd.w4 import w4_glu, w4_linear
        call = w4_linear if op == "w4_linear" else w4_glu
        return call(s["x"], s["codes"], s["scale"], s["zero"], out_dtype=DT[case["out"]])
    from mxfp4_routed_expert_gemv_amd.grads import clip_grads, grad_norm
    if op == "norm":
        return grad_norm(s["grads"])
    return clip_grads(s["grads"], s["max_norm"], out=s["outs"]), s["outs"]


def _plain(s):
    op, case = s["case"]["op"], s["case"]
    if op in ("train", "backward"):
        S, fs, d = case["S"], case["fs"], case["d"]
        x, w13 = s["x"].float(), s["w13"].float().view(S * 2 * fs, d)
        # the experts' hidden features side by side: one product over all of them is their sum
        w2 = s["w2"].float().transpose(0, 1).reshape(d, S * fs)
        T = x.shape[0]
        if op == "train":
            gu = (x @ w13.t()).view(T, S, 2 * fs)
            gate, up = gu[..., :fs], gu[..., fs:]
            h = gate / (1 + torch.exp(-gate)) * up
            return (h.reshape(T, S * fs) @ w2.t()).bfloat16(), gu.bfloat16()
        dy, gu = s["dy"].float(), s["gu"].float()
        gate, up = gu[..., :fs], gu[..., fs:]
        sig = 1 / (1 + torch.exp(-gate))
        dh = (dy @ w2).view(T, S, fs)
        dgu = torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], -1).view(T, S * 2 * fs)
        h = (gate * sig * up).view(T, S * fs)
        dw2 = (dy.t() @ h).view(d, S, fs).transpose(0, 1)
        return ((dgu @ w13).bfloat16(), (dgu.t() @ x).view(S, 2 * fs, d).bfloat16(),
                dw2.bfloat16().contiguous())
    if op in ("w4_linear", "w4_glu"):
        w = _weights(s["codes"], s["scale"], s["zero"], torch.float32)
        out = s["x"].float() @ w.t()
        if op == "w4_glu":
            f = case["n"] // 2
            out = out[:, :f] / (1 + torch.exp(-out[:, :f])) * out[:, f:]
        return out.to(DT[case["out"]])
    norm = torch.stack([t.double().square().sum() for t in s["grads"]]).sum().sqrt()
    if op == "norm":
        return norm.float()
    factor = (s["max_norm"] / norm).clamp(max=1.0).float()
    [o.copy_(t.float() * factor) for t, o in zip(s["grads"], s["outs"])]
    return norm.float(), s["outs"]


def _weights(codes, scale, zero, dtype):
    n, half = codes.shape
    q = torch.stack([codes & 15, codes >> 4], -1).view(n, scale.shape[1], -1).to(dtype)
    z = 8.0 if zero is None else zero.to(dtype)[..., None]
    return ((q - z) * scale.to(dtype)[..., None]).view(n, 2 * half)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] in ("train", "backward"):
        x = s["x"].to(f8)
        gate_w, up_w = (s["w13"].to(f8)[:, i * case["fs"]: (i + 1) * case["fs"]] for i in (0, 1))
        experts = range(case["S"])
        if case["op"] == "train":
            g, u = ([x @ w[j].t() for j in experts] for w in (gate_w, up_w))
            y = sum((g[j] * torch.sigmoid(g[j]) * u[j]) @ s["w2"][j].to(f8).t() for j in experts)
            return y, torch.stack([torch.cat([g[j], u[j]], 1) for j in experts], 1)
        dy, dx, dw13, dw2 = s["dy"].to(f8), 0, [], []
        for j in experts:
            g, u = s["gu"][:, j].to(f8).chunk(2, 1)
            sig = torch.sigmoid(g)
            dh = dy @ s["w2"][j].to(f8)
            dg, du = dh * u * (sig + g * sig * (1 - sig)), dh * g * sig
            dx = dx + dg @ gate_w[j] + du @ up_w[j]
            dw13.append(torch.cat([dg.t() @ x, du.t() @ x]))
            dw2.append(dy.t() @ (g * sig * u))
        return dx, torch.stack(dw13), torch.stack(dw2)
    if case["op"] in ("w4_linear", "w4_glu"):
        group, n, k = case["group"], case["n"], case["k"]
        byte = s["codes"].to(torch.int64)
        q = torch.empty((n, k), dtype=f8, device="cuda")
        q[:, 0::2], q[:, 1::2] = (byte % 16).to(f8), (byte // 16).to(f8)
        z = torch.full_like(s["scale"], 8.0) if s["zero"] is None else s["zero"]
        w = (q - z.to(f8).repeat_interleave(group, 1)) * s["scale"].to(f8).repeat_interleave(group, 1)
        out = s["x"].to(f8) @ w.t()
        return out if case["op"] == "w4_linear" else (
            out[:, :n // 2] * torch.sigmoid(out[:, :n // 2]) * out[:, n // 2:])
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t.to(f8))) ** 2 for t in s["grads"]))
    if case["op"] == "norm":
        return torch.tensor(norm, dtype=f8)
    factor = min(1.0, s["max_norm"] / norm)
    return torch.tensor(norm, dtype=f8), [t.to(f8) * factor for t in s["grads"]]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] in ("train", "backward"):
        T, d, F = case["T"], case["d"], case["S"] * case["fs"]
        weights = 2 * 3 * d * F
        if case["op"] == "train":
            return {"bytes": weights + 2 * T * (d + d + 2 * F), "flops": 6 * T * d * F}
        return {"bytes": 2 * weights + 2 * T * (3 * d + 2 * F), "flops": 12 * T * d * F}
    if case["op"] in ("w4_linear", "w4_glu"):
        T, n, k, group = (case[v] for v in ("T", "n", "k", "group"))
        size = {"f32": 4, "bf16": 2}
        groups = n * k // group
        outs = T * (n if case["op"] == "w4_linear" else n // 2)
        return {"bytes": n * k // 2 + groups * (3 if case["zero"] else 2) + size[case["x"]] * T * k
                + size[case["out"]] * outs, "flops": 2 * T * n * k}
    total, size = sum(_sizes(case)), 2 if case["bf16"] else 4
    write = {"f32": 4, "bf16": 2}[case["out"]] if case["op"] == "clip" else 0
    return {"bytes": total * (size + write), "flops": (2 if case["op"] == "norm" else 3) * total}
