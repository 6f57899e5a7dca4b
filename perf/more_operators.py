"""Workloads of the operators that train through the routing (routing.py) and
of the orthogonalised update of a weight matrix (ortho.py).

A case is a dict of plain values.  `run` computes one pass in plain torch
operations, or, where `own` is true, through the library's entry points;
`exact` computes the same outputs in 64 bits from the definitions.

  dispatch       rows, order = dispatch(x, idx, E): the (token, slot) pairs sorted
                 by expert, and each pair's row of x at its place
    back         dx = dispatch_backward(drows, order): a token's rows summed
  collect        y = collect(rows, order, w, add): the experts' rows back at
                 their tokens, weighted and summed (and the shared experts' y)
    back         drows, dw = collect_backward(dy, rows, order, w)
  route          dx, dw_router = route_backward(x, w_router, idx, w, dw, order, ...):
                 from the gradient of the combine weights to the router's
  orthogonalize  o = orthogonalize(g): Newton-Schulz steps p(X) = a X + b (X X^T) X
                 + c (X X^T)^2 X from X = g / |g|, the update of a Muon step

A pair whose id is outside [0, E), or an earlier slot's of its token, has no row.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIGMA = 0.02                             # standard deviation of the router's weights
STEPS, COEFFICIENTS = 5, (3.4445, -4.7750, 2.0315)


# ------------------------------------------------------------------ the cases
def _pairs(op, name, T, d, E, k, rows, out, back=False, add=False, padded=0.0, zipf=0.0,
           router="softmax"):
    return {"name": name, "op": op, "T": T, "d": d, "E": E, "k": k, "rows": rows, "out": out,
            "back": back, "add": add, "padded": padded, "zipf": zipf, "router": router}


def _ortho(name, batch, m, n, g, rank):
    return {"name": name, "op": "orthogonalize", "batch": batch, "m": m, "n": n, "g": g, "rank": rank}


def listed():
    return [
        # a handful of tokens through a toy layer: a unit test's step, all latency
        _pairs("dispatch", "dispatch, toy layer", 4, 256, 16, 4, "f32", "f32"),
        # an ordinary micro-batch of the full-size layer
        _pairs("dispatch", "dispatch, 4096 tokens", 4096, 7168, 896, 16, "bf16", "bf16"),
        # a packed batch whose last tokens are padding, gradients kept in fp32
        _pairs("dispatch", "dispatch back, 1000 tokens", 1000, 7168, 896, 16, "f32", "f32", back=True,
               padded=0.07),
        # a short ragged batch: the experts' fp32 rows onto the shared experts' result
        _pairs("collect", "collect, 37 tokens", 37, 7168, 896, 16, "f32", "bf16", add=True),
        # the largest batch that the layer is measured on, a skewed routing
        _pairs("collect", "collect, 16384 tokens", 16384, 7168, 896, 16, "bf16", "bf16", add=True,
               zipf=1.1),
        # a ragged sequence, the experts' rows as the 4-bit experts give them
        _pairs("collect", "collect back, 517 tokens", 517, 7168, 896, 16, "f32", "bf16", back=True),
        # the ordinary micro-batch
        _pairs("collect", "collect back, 4096 tokens", 4096, 7168, 896, 16, "bf16", "bf16", back=True),
        # few tokens: what the router's gradient costs beside reading and writing its weights
        _pairs("route", "route back, 64 tokens", 64, 7168, 896, 16, "bf16", "bf16", back=True,
               router="sigmoid_norm"),
        # the largest batch: popular experts have thousands of tokens, others none
        _pairs("route", "route back, 16384 tokens", 16384, 7168, 896, 16, "bf16", "f32", back=True,
               zipf=1.1),
        # the toy layer's matrix, all latency
        _ortho("orthogonalize, 256 x 128", 1, 256, 128, "f32", 4),
        # the router's gradient, wide and flat
        _ortho("orthogonalize, 896 x 7168", 1, 896, 7168, "f32", 32),
        # both shared experts' gate and up gradients
        _ortho("orthogonalize, 2 x 4096 x 7168", 2, 4096, 7168, "bf16", 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch", "collect", "collect", "route", "orthogonalize",
                     "orthogonalize"])
    if op == "orthogonalize":
        m, n = _log(rng, 12, 7168), _log(rng, 12, 7168)
        most = 2 * 4096 * 4096 * 7168 // (min(m, n) * m * n)
        c = _ortho("", min(_log(rng, 1, 12), max(1, most)), m, n, rng.choice(["f32", "bf16"]),
                   _log(rng, 1, 64))
    else:
        d = 32 * _log(rng, 4, 256)
        E = _log(rng, 4, 1024)
        k = min(_log(rng, 1, 24), E)
        T = _log(rng, 1, min(16384, 16384 * 16 * 7168 // (k * d)))
        c = _pairs(op, "", T, d, E, k, rng.choice(["f32", "bf16", "bf16"]) if T * k * d < 10 ** 9 else "bf16",
                   rng.choice(["f32", "bf16"]), back=op == "route" or rng.random() < 0.5,
                   add=rng.random() < 0.5, padded=rng.choice([0.0, 0.0, 0.1]),
                   zipf=rng.choice([0.0, 1.1]),
                   # (of one expert a token, the others' weight is always 1 and has no gradient)
                   router=rng.choice(["softmax", "sigmoid", "sigmoid_norm"] if k > 1 else ["sigmoid"]))
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g)
        return t.to(dtype)

    s = {"case": case}
    if case["op"] == "orthogonalize":
        # a gradient: some directions well over the noise, each half as strong as the one before
        # but for a floor
        B, m, n, r = (case[v] for v in ("batch", "m", "n", "rank"))
        r = min(r, m, n)
        strength = (0.5 ** torch.arange(r, device="cuda", dtype=torch.float32)).clamp(min=0.02)
        t = torch.bmm(normal(B, m, r) * strength, normal(B, r, n))
        s["g"] = (normal(B, m, n, std=0.05).add_(t, alpha=0.25) * 0.01).to(DT[case["g"]])
        if B == 1:
            s["g"] = s["g"][0]
        return s
    T, d, E, k = (case[v] for v in ("T", "d", "E", "k"))
    logits = normal(T, E, std=SIGMA * math.sqrt(7168))
    if case["zipf"]:
        # the popularity of expert e falls as (1 + e) ** -zipf, the experts in an order of their own
        place = torch.randperm(E, generator=g, device="cuda")
        logits -= case["zipf"] * torch.log1p(place.float())
    idx = logits.topk(k).indices.sort(1).values
    chosen = logits.gather(1, idx)
    if case["router"] == "softmax":
        w = torch.softmax(chosen, 1)
    else:
        w = torch.sigmoid(chosen)
        if case["router"] == "sigmoid_norm":
            w = w / w.sum(1, keepdim=True)
    idx = idx.int()
    if case["padded"]:
        idx[T - int(T * case["padded"]):] = -1
    back, rows, out = case["back"], DT[case["rows"]], DT[case["out"]]
    s["idx"], s["w"] = idx, w
    if case["op"] == "dispatch" and not back:
        s["x"] = normal(T, d, dtype=rows)
        return s
    s["order"] = _order(idx, E)
    s["pair_pos"] = s["order"][3]
    if case["op"] == "dispatch":
        s["drows"] = normal(T * k, d, std=0.01, dtype=rows)
    elif case["op"] == "collect":
        s["rows"] = normal(T * k, d, dtype=rows)
        s["dy" if back else "add"] = (normal(T, d, std=0.01 if back else 1.0, dtype=out)
                                      if back or case["add"] else None)
    else:
        s["x"] = normal(T, d, dtype=rows)
        s["w_router"] = normal(E, d, std=SIGMA, dtype=torch.bfloat16)
        s["dw"] = normal(T, k, std=0.01)
        s["logits"] = logits
    return s


def _order(idx, E):
    """counts [E], offsets [E + 1], sorted_pair [T k] and pair_pos [T][k] of ids [T][k]."""
    T, k = idx.shape
    pairs = torch.arange(T * k, device=idx.device)
    same = idx[:, :, None] == idx[:, None, :]
    earlier = torch.ones(k, k, dtype=torch.bool, device=idx.device).tril(-1)
    valid = ((idx >= 0) & (idx < E) & ~(same & earlier).any(2)).view(-1)
    key = torch.where(valid, idx.view(-1).long(), E)
    order = key.sort(stable=True).indices
    pos = torch.empty_like(order).scatter_(0, order, pairs)
    counts = torch.zeros(E + 1, dtype=torch.long, device=idx.device).scatter_add_(0, key, torch.ones_like(key))[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return (counts.int(), offsets.int(), torch.where(valid[order], order, -1).int(),
            torch.where(valid, pos, -1).int().view(T, k))


# ------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    case = s["case"]
    if case["op"] == "orthogonalize":
        from mxfp4_routed_expert_gemv_amd.ortho import orthogonalize
        return orthogonalize(s["g"], steps=STEPS, coefficients=COEFFICIENTS)
    from mxfp4_routed_expert_gemv_amd import routing
    out = DT[case["out"]]
    if case["op"] == "dispatch":
        if case["back"]:
            return routing.dispatch_backward(s["drows"], s["order"], out_dtype=out)
        rows, order = routing.dispatch(s["x"], s["idx"], case["E"])
        return (rows, *order)
    if case["op"] == "collect":
        if case["back"]:
            return routing.collect_backward(s["dy"], s["rows"], s["order"], s["w"])
        return routing.collect(s["rows"], s["order"], s["w"], add=s["add"], out_dtype=out)
    return routing.route_backward(
        s["x"], s["w_router"], s["idx"], s["w"], s["dw"], s["order"], router=case["router"],
        logits=s["logits"] if case["router"] == "sigmoid_norm" else None, dw_dtype=out)


def _plain(s):
    case = s["case"]
    if case["op"] == "orthogonalize":
        g = s["g"].float()
        m, n = g.shape[-2:]
        g = g.view(-1, m, n)
        x = g.transpose(1, 2).contiguous() if m > n else g
        norm = x.double().square().sum((1, 2), keepdim=True).sqrt()
        x = (x / norm).float()
        a, b, c = COEFFICIENTS
        for _ in range(STEPS):
            gram = torch.bmm(x, x.transpose(1, 2).contiguous())
            x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
        return (x.transpose(1, 2) if m > n else x).bfloat16().reshape(s["g"].shape)
    T, d, E, k = (case[v] for v in ("T", "d", "E", "k"))
    rows_dt, out = DT[case["rows"]], DT[case["out"]]
    if case["op"] == "dispatch" and not case["back"]:
        order = _order(s["idx"], E)
        pair = order[2].long()
        return (s["x"][pair.clamp(min=0) // k].masked_fill_((pair < 0)[:, None], 0.0), *order)
    if case["op"] == "route":
        dl, idx, x = _dlogits(s, torch.float32), s["idx"].long(), s["x"].float()
        dense = x.new_zeros(T, E + 1).scatter_add_(
            1, torch.where(s["pair_pos"] >= 0, idx, E), dl)[:, :E].contiguous()
        return (dense @ s["w_router"].float()).to(rows_dt), (dense.t() @ x).to(out)
    pos = s["pair_pos"].long()
    there = (pos >= 0)[:, :, None]
    if case["op"] == "dispatch":
        return s["drows"][pos.clamp(min=0)].float().masked_fill_(~there, 0.0).sum(1).to(out)
    rows = s["rows"][pos.clamp(min=0)].float()
    w = s["w"][:, :, None]
    if not case["back"]:
        y = rows.mul_(w).masked_fill_(~there | (w == 0), 0.0).sum(1)
        return (y if s["add"] is None else y + s["add"].float()).to(out)
    dy = s["dy"].float()[:, None, :]
    dw = rows.mul_(dy).sum(2).masked_fill_(~there[:, :, 0], 0.0)
    drows = torch.zeros(T * k + 1, d, dtype=rows_dt, device=dy.device)
    drows[torch.where(pos >= 0, pos, T * k)] = (w * dy).to(rows_dt)
    return drows[:T * k], dw


def _dlogits(s, dt):
    """The gradient of the chosen experts' logits from that of their weights."""
    router, w, dw = s["case"]["router"], s["w"].to(dt), s["dw"].to(dt)
    dw = dw.masked_fill(s["pair_pos"] < 0, 0.0)
    if router == "softmax":
        return w * (dw - (w * dw).sum(1, keepdim=True))
    if router == "sigmoid":
        return dw * w * (1 - w)
    # w = s / sum(s), s the chosen experts' sigmoids: dw_i / ds_j = ((i == j) - w_i) / sum(s)
    idx = s["idx"].long().clamp(0, s["case"]["E"] - 1)
    sig = 1 / (1 + torch.exp(-s["logits"].gather(1, idx).to(dt)))
    return w * (1 - sig) * (dw - (w * dw).sum(1, keepdim=True))


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "orthogonalize":
        a, b, c = COEFFICIENTS
        outs = []
        for g in s["g"].to(f8).view(-1, case["m"], case["n"]):
            x = g / torch.linalg.vector_norm(g)
            wide = x.shape[0] <= x.shape[1]
            for _ in range(STEPS):
                gram = x @ x.t() if wide else x.t() @ x
                poly = b * gram + c * gram @ gram
                x = a * x + (poly @ x if wide else x @ poly)
            outs.append(x)
        return torch.stack(outs).view(s["g"].shape)
    T, d, E, k = (case[v] for v in ("T", "d", "E", "k"))
    if case["op"] == "dispatch" and not case["back"]:
        pair = _order(s["idx"], E)[2].long()
        rows = torch.zeros(T * k, d, dtype=f8, device="cuda")
        rows[pair >= 0] = s["x"].to(f8)[pair[pair >= 0] // k]
        return rows, None, None, None, None
    if case["op"] == "route":
        x, wr = s["x"].to(f8), s["w_router"].to(f8)
        dx, dwr = torch.zeros_like(x), torch.zeros_like(wr)
        dl = _dlogits(s, f8)
        for e in range(0, k):   # one slot's expert for every token
            t = (s["pair_pos"][:, e] >= 0).nonzero()[:, 0]
            i, v = s["idx"][t, e].long(), dl[t, e, None]
            dx[t] += v * wr[i]
            dwr.index_add_(0, i, v * x[t])
        return dx, dwr
    pos = s["pair_pos"].long()
    if case["op"] == "dispatch":
        dx = torch.zeros(T, d, dtype=f8, device="cuda")
        for j in range(k):
            t = (pos[:, j] >= 0).nonzero()[:, 0]
            dx[t] += s["drows"][pos[t, j]].to(f8)
        return dx
    w = s["w"].to(f8)
    if not case["back"]:
        y = torch.zeros(T, d, dtype=f8, device="cuda") if s["add"] is None else s["add"].to(f8)
        for j in range(k):
            t = ((pos[:, j] >= 0) & (w[:, j] != 0)).nonzero()[:, 0]
            y[t] += w[t, j, None] * s["rows"][pos[t, j]].to(f8)
        return y
    dy, dw = s["dy"].to(f8), torch.zeros(T, k, dtype=f8, device="cuda")
    drows = torch.zeros(T * k, d, dtype=f8, device="cuda")
    for j in range(k):
        t = (pos[:, j] >= 0).nonzero()[:, 0]
        drows[pos[t, j]] = w[t, j, None] * dy[t]
        dw[t, j] = (s["rows"][pos[t, j]].to(f8) * dy[t]).sum(1)
    return drows, dw


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "orthogonalize":
        B, m, n = case["batch"], case["m"], case["n"]
        short, long = min(m, n), max(m, n)
        # a step's three products; the first two are symmetric, so half of each is needed
        step = short * short * long + short ** 3 + 2 * short * short * long
        return {"bytes": B * m * n * (size[case["g"]] + 2), "flops": STEPS * B * step}
    T, d, E, k = (case[v] for v in ("T", "d", "E", "k"))
    r, o, P = size[case["rows"]], size[case["out"]], T * k
    if case["op"] == "dispatch":
        if case["back"]:
            return {"bytes": P * (d * r + 4) + T * d * o, "flops": P * d}
        return {"bytes": T * d * r + P * (d * r + 4 + 8) + 8 * E, "flops": 0}
    if case["op"] == "collect":
        if case["back"]:
            return {"bytes": T * d * o + P * (2 * d * r + 12), "flops": 3 * P * d}
        return {"bytes": P * (d * r + 8) + T * d * o * (2 if case["add"] else 1), "flops": 2 * P * d}
    return {"bytes": 2 * T * d * r + E * d * (2 + o) + P * 16, "flops": 4 * P * d}
