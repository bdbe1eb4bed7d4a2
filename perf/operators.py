"""Cases of the operators that train a Mixture-of-Experts feed-forward sublayer.

Five operators, in the order a backward pass meets them:

  norm   layer norm in front of the router: forward, and its backward pass with
         the reduction of the weight's and the bias's gradients over the tokens
  ffn    the experts' gated feed-forward block on rows grouped by expert: both
         projections, the activation and the product, then the down projection
         and the weighted combine; what the backward pass needs is kept
  grad   its backward pass: the gradients of the rows and of all three weights
  rows   the gradients around the experts: of the weighted combine (rows and
         top-K weights) and of the dispatch (rows back to tokens)
  route  the router's backward pass: top-K softmax, balance and z-loss terms,
         the tokens' gradient (summed with the rows that come back from the
         experts) and the router weight's

Each case is one call as a training step makes it.  ``run`` computes it in
elementary torch operations in 32 bits, or, with ``own`` set, by the library's
kernels.
"""
import math

import torch

own = False

EPS = 1e-5
BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32


def listed():
    return [
        # the norm of a decode-sized batch: launch latency
        {"name": "norm_decode", "op": "norm", "T": 256, "d": 4096, "dtype": "bf16", "backward": False},
        # forward and backward of a training step's norm, the residual's gradient added
        {"name": "norm_step", "op": "norm", "T": 16384, "d": 4096, "dtype": "bf16", "backward": True},
        # a residual stream kept in 32 bits, an odd number of tokens
        {"name": "norm_fp32_odd", "op": "norm", "T": 4099, "d": 7168, "dtype": "fp32", "backward": True},
        # experts' forward: a decode-sized batch (the weights' stream bounds it), a full training batch, many small experts
        {"name": "ffn_few_rows", "op": "ffn", "T": 256, "d": 4096, "f": 14336, "E": 8, "K": 2, "drop": 0.0},
        {"name": "ffn_batch", "op": "ffn", "T": 16384, "d": 4096, "f": 14336, "E": 8, "K": 2, "drop": 0.0},
        # experts' backward: the smallest layer (latency), 60 small experts with dropped slots, the full batch
        {"name": "grad_tiny", "op": "grad", "T": 64, "d": 128, "f": 256, "E": 8, "K": 2, "drop": 0.0},
        {"name": "grad_small_experts", "op": "grad", "T": 8192, "d": 2048, "f": 1408, "E": 60, "K": 4, "drop": 0.25},
        {"name": "grad_batch", "op": "grad", "T": 16384, "d": 4096, "f": 14336, "E": 8, "K": 2, "drop": 0.0},
        # gradients of combine and dispatch: a small batch, and one with a quarter of the slots dropped
        {"name": "rows_few", "op": "rows", "T": 256, "d": 4096, "E": 8, "K": 2, "drop": 0.0},
        {"name": "rows_dropped", "op": "rows", "T": 8192, "d": 2048, "E": 60, "K": 4, "drop": 0.25},
        # router's backward: few experts and many tokens, 256 experts and wide tokens
        {"name": "route_8", "op": "route", "T": 16384, "d": 4096, "E": 8, "K": 2, "drop": 0.0},
        {"name": "route_256", "op": "route", "T": 4096, "d": 7168, "E": 256, "K": 8, "drop": 0.0},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "ffn", "grad", "rows", "route"])
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 16384), "d": _log(rng, 64, 7168, 16), "dtype": rng.choice(["bf16", "fp32"]),
                "backward": rng.random() < 0.7}
    if op in ("rows", "route"):
        E = rng.choice([1, 3, 8, 17, 60, 64, 128, 256])
        return {"op": op, "T": _log(rng, 1, 8192), "d": _log(rng, 64, 7168, 16), "E": E, "K": rng.randint(1, min(E, 8)),
                "drop": rng.choice([0.0, 0.0, 0.25])}
    while True:
        E = rng.choice([1, 2, 7, 8, 16, 60, 64])
        T, K = _log(rng, 1, 16384), rng.randint(1, min(E, 8))
        d, f = _log(rng, 64, 7168, 16), _log(rng, 64, 14336, 16)
        if T * K * d * f <= 3e11 and E * d * f <= 5e8:
            return {"op": op, "T": T, "d": d, "f": f, "E": E, "K": K, "drop": rng.choice([0.0, 0.0, 0.25])}


# ---------------------------------------------------------------- inputs

def _normal(g, shape, std, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _routing(case, g):
    """K distinct experts a token, uneven popularity, a share of the slots dropped;
    the kept slots' rows grouped by expert in token order."""
    T, E, K = case["T"], case["E"], case["K"]
    score = torch.rand((T, E), generator=g, device="cuda") + 0.3 * torch.rand(E, generator=g, device="cuda")
    val, idx = score.topk(K, dim=1)
    flat = idx.reshape(-1).clone()
    n = T * K - int(case["drop"] * T * K)
    flat[torch.rand(T * K, generator=g, device="cuda").argsort()[n:]] = E
    order = flat.argsort(stable=True)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    inv = torch.full((T * K,), -1, device="cuda", dtype=I32)
    inv[order[:n]] = torch.arange(n, device="cuda", dtype=I32)
    offsets = torch.zeros(E + 1, device="cuda", dtype=I32)
    offsets[1:] = counts.cumsum(0)
    return {"n": n, "most": int(counts.max()), "topk_idx": idx.to(I32), "topk_w": torch.softmax(4 * val, 1), "inv": inv.view(T, K),
            "offsets": offsets, "counts": torch.bincount(idx.reshape(-1), minlength=E).to(I32)}


def _scratch_bytes(case):
    """Room for any of the library's workspaces at these sizes."""
    if case["op"] == "norm":
        return 4096 + 8 * 320 * case["d"]
    if case["op"] == "route":
        e = -(-case["E"] // 64) * 64
        return 8192 + 2 * e * (case["T"] + case["d"]) + 4 * 16 * e * case["d"]
    return 4096


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, d = case["T"], case["d"]
    empty = lambda *shape, dtype=BF16: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    s = {"case": case, "ws": torch.zeros(_scratch_bytes(case), dtype=torch.uint8, device="cuda")}
    if case["op"] == "norm":
        t = BF16 if case["dtype"] == "bf16" else F32
        s.update(x=_normal(g, (T, d), 1.5, t).add_(0.25), gamma=1 + _normal(g, (d,), 0.1, F32), beta=_normal(g, (d,), 0.1, F32),
                 dy=_normal(g, (T, d), 1e-2, t), dx_add=_normal(g, (T, d), 1e-2, t))
        s.update(y=empty(T, d, dtype=t), mean=empty(T, dtype=F32), rstd=empty(T, dtype=F32), dx=empty(T, d, dtype=t),
                 dgamma=empty(d, dtype=F32), dbeta=empty(d, dtype=F32))
        return s
    E, K = case["E"], case["K"]
    s.update(_routing(case, g))
    A = T * K
    if case["op"] in ("ffn", "grad"):
        f = case["f"]
        s.update(x_perm=_normal(g, (A, d), 1.0), W1=_normal(g, (E, d, f), d ** -0.5), W3=_normal(g, (E, d, f), d ** -0.5),
                 W2=_normal(g, (E, f, d), f ** -0.5))
        if case["op"] == "ffn":
            s.update(gu=empty(A, 2 * f), h=empty(A, f), y_perm=empty(A, d, dtype=F32), y=empty(T, d))
        else:
            gu = _normal(g, (A, 2 * f), 1.0)
            a = gu[:, :f].float()
            h = (a * torch.sigmoid(a) * gu[:, f:].float()).to(BF16)
            s.update(gu=gu, h=h, dy_perm=_normal(g, (A, d), 1e-2), dgu=empty(A, 2 * f), dx_perm=empty(A, d), dW1=empty(E, d, f),
                     dW3=empty(E, d, f), dW2=empty(E, f, d))
    elif case["op"] == "rows":
        s.update(dy=_normal(g, (T, d), 1e-2), y_perm=_normal(g, (A, d), 1.0, F32), dx_perm=_normal(g, (A, d), 1e-2))
        s.update(dy_perm=empty(A, d), dtopk_w=empty(T, K, dtype=F32), dx=empty(T, d))
    else:
        s.update(x=_normal(g, (T, d), 1.0), Wr=_normal(g, (d, E), d ** -0.5), logits=_normal(g, (T, E), 1.0, F32),
                 dtopk_w=_normal(g, (T, K), 1e-2, F32), dx_perm=_normal(g, (A, d), 1e-3))
        s.update(dx=empty(T, d), dWr=empty(d, E), dlogits=empty(T, E, dtype=F32))
    return s


AUX, ZL = 0.01, 0.001  # what the loss weighs the balance loss and the z-loss with


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"norm": _norm, "ffn": _ffn, "grad": _grad, "rows": _rows, "route": _route}[op](s)


def _own(op, s):
    from moe_layer_gemm_b200 import abi

    c = s["case"]
    if op == "norm":
        abi.moe_layernorm(s["x"], s["gamma"], s["beta"], EPS, s["y"], s["mean"], s["rstd"])
        out = {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
        if c["backward"]:
            abi.moe_layernorm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dx_add"], s["dx"], s["dgamma"], s["dbeta"], s["ws"])
            out.update(dx=s["dx"], dgamma=s["dgamma"], dbeta=s["dbeta"])
        return out
    dims, n = abi.Dims(c["T"], c["d"], c.get("f", 16), c["E"], c["K"]), s["n"]
    if op == "ffn":
        abi.moe_ffn_train(dims, s["x_perm"], s["offsets"], s["W1"], s["W3"], s["W2"], s["gu"], s["h"], s["y_perm"], s["ws"])
        abi.moe_combine(dims, s["y_perm"], s["inv"], s["topk_w"], s["y"])
        return {"gu": s["gu"][:n], "h": s["h"][:n], "y": s["y"]}
    if op == "grad":
        abi.moe_ffn_backward(dims, s["dy_perm"], s["x_perm"], s["offsets"], s["W1"], s["W3"], s["W2"], s["gu"], s["h"], s["dgu"], s["dx_perm"],
                             s["dW1"], s["dW3"], s["dW2"], s["ws"])
        return {"dgu": s["dgu"][:n], "dx_perm": s["dx_perm"][:n], "dW1": s["dW1"], "dW3": s["dW3"], "dW2": s["dW2"]}
    if op == "rows":
        abi.moe_combine_backward(dims, s["dy"], s["y_perm"], s["inv"], s["topk_w"], s["dy_perm"], s["dtopk_w"])
        abi.moe_permute_backward(dims, s["dx_perm"], s["inv"], s["dx"])
        return {"dy_perm": s["dy_perm"][:n], "dtopk_w": s["dtopk_w"], "dx": s["dx"]}
    abi.moe_route_backward(dims, s["x"], s["Wr"], s["logits"], s["topk_idx"], s["topk_w"], s["dtopk_w"], s["counts"], AUX, ZL, s["dx_perm"],
                           s["inv"], s["dx"], s["dWr"], s["dlogits"], s["ws"])
    return {"dx": s["dx"], "dWr": s["dWr"], "dlogits": s["dlogits"]}


def _norm(s):
    x, t = s["x"].float(), s["x"].dtype
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = torch.rsqrt((xc * xc).mean(1) + EPS)
    xhat = xc * rstd[:, None]
    out = {"y": (xhat * s["gamma"] + s["beta"]).to(t), "mean": mean, "rstd": rstd}
    if s["case"]["backward"]:
        dy = s["dy"].float()
        q = dy * s["gamma"]
        dx = rstd[:, None] * (q - q.mean(1, keepdim=True) - xhat * (q * xhat).mean(1, keepdim=True))
        out.update(dx=(dx + s["dx_add"].float()).to(t), dgamma=(dy * xhat).sum(0), dbeta=dy.sum(0))
    return out


def _slots(s):
    """The slot (t, k) of each kept row."""
    inv, A = s["inv"].reshape(-1).long(), s["inv"].numel()
    at = torch.zeros(A + 1, dtype=torch.long, device=inv.device)
    at.scatter_(0, torch.where(inv < 0, A, inv), torch.arange(A, device=inv.device))
    return at[: s["n"]]


def _by_expert(s):
    """[E, most] rows of each expert, the row behind the last one where it has fewer; and each row's place in that table."""
    off, n, most = s["offsets"].long(), s["n"], s["most"]
    k = torch.arange(most, device=off.device)
    table = torch.where(k[None] < (off[1:] - off[:-1])[:, None], off[:-1, None] + k[None], n)
    r = torch.arange(n, device=off.device)
    e = torch.searchsorted(off[1:], r, right=True)
    return table, e * most + r - off[e]


def _grouped(a, n, table):
    """[E, most, width] in 32 bits, zeros where an expert has no row."""
    return torch.cat([a[:n].float(), torch.zeros_like(a[:1], dtype=F32)])[table]


def _ffn(s):
    n, (table, place) = s["n"], _by_expert(s)
    flat = lambda t: t.reshape(-1, t.shape[-1])[place]  # noqa: E731
    x = _grouped(s["x_perm"], n, table)
    g, u = torch.bmm(x, s["W1"].float()), torch.bmm(x, s["W3"].float())
    h = g * torch.sigmoid(g) * u
    y_perm = torch.cat([flat(torch.bmm(h, s["W2"].float())), torch.zeros((1, x.shape[-1]), device=x.device)])
    inv = s["inv"].long()
    y = (s["topk_w"][:, :, None] * y_perm[torch.where(inv < 0, n, inv)]).sum(1)
    return {"gu": torch.cat([flat(g), flat(u)], 1).to(BF16), "h": flat(h).to(BF16), "y": y.to(BF16)}


def _grad(s):
    n, f, (table, place) = s["n"], s["case"]["f"], _by_expert(s)
    flat = lambda t: t.reshape(-1, t.shape[-1])[place]  # noqa: E731
    dy, gu = _grouped(s["dy_perm"], n, table), _grouped(s["gu"], n, table)
    g, u = gu[..., :f], gu[..., f:]
    dh = torch.bmm(dy, s["W2"].float().transpose(1, 2))
    sg = torch.sigmoid(g)
    dg, du = dh * u * sg * (1 + g * (1 - sg)), dh * g * sg
    dx = torch.bmm(dg, s["W1"].float().transpose(1, 2)) + torch.bmm(du, s["W3"].float().transpose(1, 2))
    xt = _grouped(s["x_perm"], n, table).transpose(1, 2)
    return {"dgu": torch.cat([flat(dg), flat(du)], 1).to(BF16), "dx_perm": flat(dx).to(BF16), "dW1": torch.bmm(xt, dg).to(BF16),
            "dW3": torch.bmm(xt, du).to(BF16), "dW2": torch.bmm(_grouped(s["h"], n, table).transpose(1, 2), dy).to(BF16)}


def _back(s):
    """Tokens' sums of the rows that their kept slots own."""
    n, inv = s["n"], s["inv"].long()
    rows = torch.cat([s["dx_perm"][:n].float(), torch.zeros_like(s["dx_perm"][:1], dtype=F32)])
    return rows[torch.where(inv < 0, n, inv)].sum(1)


def _rows(s):
    n, K, at = s["n"], s["case"]["K"], _slots(s)
    dy = s["dy"].float()[at // K]
    dw = torch.zeros(s["inv"].numel(), device=at.device)
    dw[at] = (dy * s["y_perm"][:n]).sum(1)
    return {"dy_perm": (dy * s["topk_w"].reshape(-1)[at][:, None]).to(BF16), "dtopk_w": dw.view_as(s["topk_w"]), "dx": _back(s).to(BF16)}


def _route(s):
    T, E, K = s["case"]["T"], s["case"]["E"], s["case"]["K"]
    p, w, dw = torch.softmax(s["logits"], 1), s["topk_w"], s["dtopk_w"]
    fe = s["counts"].float() / (T * K)
    dl = AUX * E / T * p * (fe - (p * fe).sum(1, keepdim=True)) + ZL * 2 / T * torch.logsumexp(s["logits"], 1, keepdim=True) * p
    dl = dl.scatter_add(1, s["topk_idx"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    return {"dx": (_back(s) + dl @ s["Wr"].float().T).to(BF16), "dWr": (s["x"].float().T @ dl).to(BF16), "dlogits": dl}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    T, d = case["T"], case["d"]
    if case["op"] == "norm":
        b = 2 if case["dtype"] == "bf16" else 4
        # x in, y out, statistics; backward: dy and the added gradient in, dx out (x is read once for both)
        passes, small = (5, 8 * T + 16 * d) if case["backward"] else (2, 8 * T + 8 * d)
        return {"bytes": passes * T * d * b + small, "flops": (24 if case["backward"] else 8) * T * d}
    E, K = case["E"], case["K"]
    n = T * K - int(case["drop"] * T * K)
    if case["op"] == "ffn":
        f = case["f"]
        used = min(E, n)  # experts whose weights are read
        return {"bytes": 2 * (3 * used * d * f + n * d + 3 * n * f + T * d) + 8 * T * K, "flops": 6 * n * d * f}
    if case["op"] == "grad":
        f, used = case["f"], min(E, n)
        return {"bytes": 2 * (3 * used * d * f + 3 * E * d * f + 3 * n * d + 5 * n * f), "flops": 12 * n * d * f}
    if case["op"] == "rows":
        return {"bytes": 2 * T * d + 4 * n * d + 2 * n * d + 2 * n * d + 2 * T * d + 12 * T * K, "flops": 4 * n * d}
    return {"bytes": 2 * T * d + 2 * n * d + 2 * T * d + 4 * d * E + 8 * T * E + 16 * T * K, "flops": 4 * T * E * d + n * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    """Each operator from its formulas in 64 bits, expert by expert."""
    s = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op == "norm":
        x = s["x"].to(F64)
        var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
        sd = (var + EPS).sqrt()
        z = (x - mean) / sd
        out = {"y": z * s["gamma"].to(F64) + s["beta"].to(F64), "mean": mean[:, 0], "rstd": 1 / sd[:, 0]}
        if case["backward"]:
            dy = s["dy"].to(F64)
            dz = dy * s["gamma"].to(F64)
            d = x.shape[1]
            dx = (d * dz - dz.sum(1, keepdim=True) - z * (dz * z).sum(1, keepdim=True)) / (d * sd)
            out.update(dx=s["dx_add"].to(F64) + dx, dgamma=torch.einsum("td,td->d", dy, z), dbeta=torch.einsum("td->d", dy))
        return out
    n, off = s["n"], s["offsets"].tolist()
    inv = s["inv"].long()
    kept = (inv >= 0).to(F64)
    take = inv.clamp(min=0)

    def to_tokens(rows, w):
        out = torch.zeros((T, rows.shape[1]), dtype=F64, device="cuda")
        for k in range(case["K"]):
            if n:
                out += (w[:, k] * kept[:, k])[:, None] * rows[take[:, k]].to(F64)
        return out

    if op == "ffn":
        f = case["f"]
        gu = torch.empty((n, 2 * f), dtype=F64, device="cuda")
        h, y = torch.empty((n, f), dtype=F64, device="cuda"), torch.empty((n, case["d"]), dtype=F64, device="cuda")
        for e in range(case["E"]):
            r = slice(off[e], off[e + 1])
            x = s["x_perm"][r].to(F64)
            gu[r, :f], gu[r, f:] = x @ s["W1"][e].to(F64), x @ s["W3"][e].to(F64)
            h[r] = gu[r, :f] / (1 + torch.exp(-gu[r, :f])) * gu[r, f:]
            y[r] = h[r] @ s["W2"][e].to(F64)
        return {"gu": gu, "h": h, "y": to_tokens(y, s["topk_w"].to(F64))}
    if op == "grad":
        f, d, E = case["f"], case["d"], case["E"]
        new = lambda *shape: torch.empty(shape, dtype=F64, device="cuda")  # noqa: E731
        dgu, dx, dW1, dW3, dW2 = new(n, 2 * f), new(n, d), new(E, d, f), new(E, d, f), new(E, f, d)
        for e in range(E):
            r = slice(off[e], off[e + 1])
            x, dy, g, u = s["x_perm"][r].to(F64), s["dy_perm"][r].to(F64), s["gu"][r, :f].to(F64), s["gu"][r, f:].to(F64)
            dh, sig = dy @ s["W2"][e].to(F64).T, 1 / (1 + torch.exp(-g))
            dgu[r, :f] = dh * u * (sig + g * sig * torch.exp(-g) / (1 + torch.exp(-g)))
            dgu[r, f:] = dh * g * sig
            dx[r] = dgu[r, :f] @ s["W1"][e].to(F64).T + dgu[r, f:] @ s["W3"][e].to(F64).T
            dW1[e], dW3[e], dW2[e] = x.T @ dgu[r, :f], x.T @ dgu[r, f:], s["h"][r].to(F64).T @ dy
        return {"dgu": dgu, "dx_perm": dx, "dW1": dW1, "dW3": dW3, "dW2": dW2}
    ones = torch.ones_like(kept)
    if op == "rows":
        dy, w, K = s["dy"].to(F64), s["topk_w"].to(F64), case["K"]
        dy_perm, dw = torch.zeros((n, case["d"]), dtype=F64, device="cuda"), torch.zeros((T, K), dtype=F64, device="cuda")
        for k in range(K):
            live = (inv[:, k] >= 0).nonzero()[:, 0]
            r = inv[live, k]
            dy_perm[r] = w[live, k, None] * dy[live]
            dw[live, k] = torch.einsum("rd,rd->r", dy[live], s["y_perm"][r].to(F64))
        return {"dy_perm": dy_perm, "dtopk_w": dw, "dx": to_tokens(s["dx_perm"], ones)}
    l, w, dw, E, K = s["logits"].to(F64), s["topk_w"].to(F64), s["dtopk_w"].to(F64), case["E"], case["K"]
    lse = torch.logsumexp(l, 1, keepdim=True)
    p = torch.exp(l - lse)
    load = s["counts"].to(F64) / (T * K)
    dP = torch.full_like(p, 1 / T) * load * (AUX * E)  # of every probability
    dl = p * (dP - (dP * p).sum(1, keepdim=True)) + 2 * ZL / T * lse * p
    for k in range(K):
        term = w[:, k] * (dw[:, k] - (w * dw).sum(1))
        dl[torch.arange(T, device="cuda"), s["topk_idx"][:, k].long()] += term
    return {"dx": to_tokens(s["dx_perm"], ones) + dl @ s["Wr"].to(F64).T, "dWr": s["x"].to(F64).T @ dl, "dlogits": dl}
